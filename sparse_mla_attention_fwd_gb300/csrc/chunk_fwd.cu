// Dense MLA attention of a chunk of new tokens over a paged latent cache (sm_103a).
//
// Request b has q_b new tokens (rows cu[b] .. cu[b+1]-1 of q) and L_b keys in the cache, its new
// tokens' own rows among them.  Token i of the request stands at position L_b - q_b + i and sees
// the keys at positions j <= that (causal) or every j < L_b.  With K = row[:d_qk], V = row[:512]:
//   s_j = sm_scale <q, K_j>, m = max s_j, l = sum exp(s_j - m),
//   O = sum exp(s_j - m) V_j / (l + [sink] exp(sink_h - m)), lse = m + ln l, max_logits = m.
//
// All heads of a token, and all tokens of a request, read the same rows, so (token, head) pairs are
// simply rows of one matrix: a tile is 128 of them (whole tokens of one request, or 128 heads of one
// token when there are more).  O of a tile is 128 x 512 fp32: all of one SM's tensor memory.  So a
// PAIR of CTAs (a cluster of two, tcgen05 cta_group::2) holds a tile, 64 rows each, which leaves each
// SM half its tensor memory for scores and, unlike a 64-row tile on one SM, keeps the tensor unit's
// full width: every product is M = 128 over the pair.  Per block of 64 keys:
//   S[128 x 64]   = Q K^T     N = 64: each CTA supplies 32 keys (all d_qk columns)
//   O[128 x 512] += P V       2 x N = 256: each CTA supplies 256 value columns (all 64 keys)
// Both products find their operands at the same shared-memory offsets in both CTAs.  CTA r's 32 keys
// lie there as [D0 | D1 | rope] (columns 0-255, 256-511, 512-575).  For P V it needs, of its own
// keys, the columns of half r, where they already are, and of the other CTA's keys the same columns:
// these go into D(1-r), whose contents only S needed ("foreign" half), once S is done.  So a row's bytes
// are loaded 1.44 times per pair instead of twice, and no operand is held twice.
//
// Tensor memory of a CTA (128 lanes; row r of the CTA's 64 in lanes r and r + 64): O in columns
// 0-255 (value columns 0-255 in lanes 0-63, 256-511 in lanes 64-127), S of block b in columns
// 256 + 32 (b % 4) (keys 0-31 in lanes 0-63, 32-63 in lanes 64-127).
//
// Warps: 0 scheduler, 1 K loads, 2 foreign-half and Q loads, 3 S issuer, 4-7 softmax, 8-11 epilogue
// (both on TMEM lane quadrants 0-3), 12 PV issuer; the issuers work in the pair's first CTA.  Four buffers of
// keys: S runs up to three blocks ahead of P V, so the second load of a block and the softmax have one to
// two blocks' time.
//
// Work split.  Tiles times key blocks are laid out on one axis, a tile's cost being its keys plus a
// constant for its start and end, and the axis is cut into equal ranges, one per pair: a long
// request is spread over many pairs, short ones share one.  Every CTA finds its own range from the
// lengths with closed-form sums (no host step, no planning launch).  A tile that lies in one range is
// finished there; parts of a cut tile go to the workspace (at most two per pair) and a second
// kernel joins them.  Nothing depends on timing, so results are the same bits from call to call.
//
// The same kernel attends for trees of drafted tokens (TREE): a token sees all keys in front of its request's new ones, and the
// new ones that its row of a bit mask names.  There the axis is that of the form without causality, and four neighbouring pairs
// share their ranges tile by tile.
//
// What bounds it.  A block takes 1412 cycles of the tensor unit at full rate (36 products of N = 64, which the
// operands' 3 KB at 128 bytes a cycle of shared memory hold at 25 cycles instead of 16, and 8 of N = 256 at 64).
// Arriving keys (52 KB) and P want the same shared memory: 1690 cycles if nothing ran beside the products.  The
// L2 delivers 52 KB in 1400 (37 bytes a cycle and SM when all SMs load).  4 x 512 tokens behind 2048-8192 keys, 64
// heads: 1676 cycles a block over the whole launch, 0.94-0.96 ms = 1425-1460 TFLOP/s, L2 to SM 9.7 TB/s; 2048
// tokens over 8192 keys, 128 heads: 2.79-2.83 ms = 1445-1465 TFLOP/s; 256 tokens of one request each over 1024-4096
// keys, 128 heads: 163-166 us = 5.0 TB/s, of which 25 us are neither keys, tile ends, start nor joining.  Blocks of 128 keys (less operand traffic, two buffers instead of four) ran at the
// same pace on chunks and 12 % slower on single tokens.  Requesting keys two to eight blocks ahead into L2
// made single tokens 6 to 20 % slower.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/sparse_mla.h"
#include "host_util.cuh"
#include "pair_ptx.cuh"

namespace smla {
namespace {

constexpr int kDv = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.0f;      // O is rescaled only when a row's maximum grows by > 2^8
constexpr uint64_t kWaitLimitNs = 2000000000ull;   // every device wait gives up after 2 s

constexpr int kTileRows = 128;            // rows of a tile, 64 per CTA
constexpr int kKeys = 64;                 // keys of a block, 32 per CTA
constexpr int kGens = 4;                  // key buffers, S buffers
constexpr int kRing = 4;                  // block descriptors ahead
constexpr int kPairThreads = 416;
constexpr int kMaxPairs = 80;             // ranges the axis is cut into, at most
// Start and end of a tile, in keys (two blocks' time measured between tiles; 128 to 512 differ by 1 % on 256
// requests), and the shortest range: many parts of a tile cost more to join than longer ones to walk (one
// token over 1500 keys: 128 17.4 us, 256 15.8 us, 320 16.2 us).  kMinRange is at least kKeys, so that every
// pair between a cut tile's ends has a part of it.
constexpr int kTileCost = 192;
constexpr int kMinRange = 256;
constexpr int kTreeGroup = 4;             // neighbouring pairs that share a range in the tree form
constexpr uint32_t kHalfBytes = 16384;    // 32 keys x 256 columns
constexpr uint32_t kPBytes = 8192;        // 64 rows x 64 keys
constexpr uint32_t kTmemCols = 512, kTmemS = 256;

enum : uint32_t { kFirst = 1u, kLast = 2u, kEnd = 4u };
// Named barriers 1, 2: softmax warps that share rows; kTileBar and on, in turn: a tile is done; kAgreeBar: all
// softmax warps hand over a tile, or leave.  A wait on a named barrier has no time limit, so every one of these has to
// complete whatever wait gave up, and when.  The softmax warps leave together (agreed on once a tile), so that all of them
// have arrived for the same tiles.  The end's arrival then needs the epilogue past the barrier of the turn before, kTileBars
// tiles back: with three it is, since the last tile handed over waited for PV of the one before, and that for the epilogue
// of the one before it.
constexpr uint32_t kTileBars = 3;
constexpr uint32_t kTileBar = 3, kAgreeBar = kTileBar + kTileBars;

__device__ int g_chunk_status = 0;        // SMLA_ERR_DEVICE_TIMEOUT once any wait gave up

struct ChunkParams {
  const int32_t* block_table;
  const int32_t* cu_seqlens_q;
  const int32_t* seqlens_k;
  const float* attn_sink;   // or null
  __nv_bfloat16* out;
  float* lse;
  float* max_logits;
  float* part_o;            // [2 pairs][128 column quads][row_cap][4] unnormalised O of a tile's part
  float* part_stats;        // [2 pairs][3][128]: offset (log2 units), sum, maximum score
  int4* joins;              // [pairs]: first row, rows, last pair of the cut tile that starts there, pairs behind it without a part (bits)
  int64_t pool_rows, n_req, n_tok;
  float sm_scale;
  int h_q, max_blocks, page_block, causal;
  int box;                  // rows of a tiled load: 32, 16 or 8, a divisor of page_block; or 0
  int pool_end;             // first row behind the pool
  int tokens_per_tile, groups;   // 128 / h_q and 1, or 1 and the 128-head groups of a token
  int row_cap;
  const int32_t* tree_mask;      // [n_tok, mask_words], the tree form alone
  int mask_words;
};

// ------------------------------------------------------------------------ lengths and the axis
struct Request {
  int64_t q0, n_q, n_k, keys;   // first row token, tokens, length, readable keys
};

__device__ __forceinline__ Request request(const ChunkParams& p, int64_t b) {
  Request r;
  const int64_t c0 = __ldg(p.cu_seqlens_q + b), c1 = __ldg(p.cu_seqlens_q + b + 1);
  r.q0 = min(max(c0, static_cast<int64_t>(0)), p.n_tok);
  r.n_q = min(max(c1, r.q0), p.n_tok) - r.q0;
  r.n_k = max(__ldg(p.seqlens_k + b), 0);
  r.keys = min(r.n_k, static_cast<int64_t>(p.max_blocks) * p.page_block);
  return r;
}

__device__ __forceinline__ int64_t token_tiles(const ChunkParams& p, const Request& r) {
  return (static_cast<uint32_t>(r.n_q) + p.tokens_per_tile - 1u) / static_cast<uint32_t>(p.tokens_per_tile);
}

// Axis length of the first k token tiles of a request.  A tile's own length is at least its keys: with fewer
// keys than tokens the axis counts the tokens.
__device__ __forceinline__ int64_t axis_of(const ChunkParams& p, const Request& r, int64_t k, int64_t n) {
  if (!p.causal) return p.groups * k * (r.n_k + kTileCost);
  const int64_t base = max(r.n_k - r.n_q, static_cast<int64_t>(0)), t = p.tokens_per_tile;
  const int64_t ends = k < n ? t * (k * (k + 1) / 2) : t * (n * (n - 1) / 2) + r.n_q;   // sum of min(n_q, (i + 1) t)
  return p.groups * (k * (base + kTileCost) + (k > 0 ? ends : 0));
}
__device__ __forceinline__ int64_t axis_of(const ChunkParams& p, const Request& r) {   // the whole request
  const int64_t n = token_tiles(p, r);
  return axis_of(p, r, n, n);
}

// Length of a pair's range.
__device__ __forceinline__ int64_t range_of(int64_t total, int64_t pairs) {
  const int64_t up = total + pairs - 1;
  const int64_t each = up <= UINT32_MAX ? static_cast<uint32_t>(up) / static_cast<uint32_t>(pairs) : up / pairs;
  return max(each, static_cast<int64_t>(kMinRange));
}

// ------------------------------------------------------------------------ shared memory
struct __align__(16) BlockDesc {
  int32_t rows[kKeys];   // pool row of each key, -1 where it does not count
  uint32_t mask[2];      // validity of keys 0-31 / 32-63
  uint32_t flags;
  int32_t key0;          // position of the block's first key
  int32_t q_row, n_rows; // tile: first (token, head) row, rows
  int32_t pos0;          // position of the tile's first token; TREE: of its request's first new one
  int32_t key_end;       // keys of the tile
  int32_t part;          // workspace slot, or -1: the whole tile is done here
};

struct Control {
  BlockDesc ring[kRing];
  float ex[2][128];      // row maxima (at a tile's end row sums) of the two key halves
  float inv[2][64];      // a finished tile's factor of each row, 0 for an empty row; by tile parity
  struct {
    int32_t q_row, n_rows, part, last;   // last: the tile's last block, or -1 behind the last tile
  } done[kTileBars];
  uint64_t ring_full[kRing], ring_empty[kRing];
  uint64_t k_full[kGens], x_full[kGens];      // both CTAs' keys / foreign halves have landed (first CTA)
  uint64_t s_full[kGens], pv_done[kGens];     // S computed / PV done (both CTAs)
  uint64_t p_full, o_free, q_full;            // first CTA
  uint32_t tmem_slot;
  int abort_flag;
};

struct RangeScan {       // lies in the P tile until the first P is written
  int64_t warp_sum[kPairThreads / 32];
  int64_t total, run;
  int64_t req, start;    // request in which this pair's range starts, its position on the axis
};

template <int D_QK>
struct Smem {
  static constexpr int kChunks = D_QK / 64;
  static constexpr uint32_t kQBytes = 64 * D_QK * 2;
  static constexpr uint32_t kGenBytes = 32 * D_QK * 2;
  static constexpr uint32_t kP = kQBytes + kGens * kGenBytes;
  static constexpr uint32_t kControl = kP + kPBytes;
  static constexpr uint32_t kBytes = kControl + sizeof(Control);
};
static_assert(Smem<576>::kBytes <= 232448, "a CTA's shared memory");

// Lane i of four neighbours holds pieces 0-3 of row i; afterwards piece i of rows 0-3.
__device__ __forceinline__ void transpose_4x4(uint32_t (&v)[4][4], int lane) {
  const bool hi2 = lane & 2, hi1 = lane & 1;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, hi2 ? v[x][w] : v[x + 2][w], 2);
      if (hi2) v[x][w] = got;
      else v[x + 2][w] = got;
    }
#pragma unroll
    for (int x = 0; x < 4; x += 2) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, hi1 ? v[x][w] : v[x + 1][w], 1);
      if (hi1) v[x][w] = got;
      else v[x + 1][w] = got;
    }
  }
}

// ------------------------------------------------------------------------ bounded waits
__device__ __forceinline__ void give_up(volatile int* abort) {
  *abort = 1;
  atomicExch(&g_chunk_status, static_cast<int>(SMLA_ERR_DEVICE_TIMEOUT));
}

// The clock and the abort flag are looked at every 16 tries: with both in every try the kernel is 2 % slower.
template <bool PAIR>
__device__ __forceinline__ void wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort,
                                             uint64_t limit_ns = kWaitLimitNs) {
  constexpr uint32_t kSleepNs = 100000;
  const uint32_t a = smem_u32(bar);
  auto done = [&] { return PAIR ? mbar_sleep_cluster(a, parity, kSleepNs) : mbar_sleep(a, parity, kSleepNs); };
  if (done()) return;
  const uint64_t t0 = globaltimer_ns();
  uint32_t tries = 0;
  while (!done())
    if ((++tries & 15u) == 0u && (*abort || globaltimer_ns() - t0 > limit_ns)) return give_up(abort);
}
__device__ __forceinline__ void wait_on(uint64_t* bar, uint32_t parity, volatile int* abort) {
  wait_bounded<false>(bar, parity, abort);
}
// For a barrier on which the other CTA's threads arrive.
__device__ __forceinline__ void wait_on_pair(uint64_t* bar, uint32_t parity, volatile int* abort) {
  wait_bounded<true>(bar, parity, abort);
}

// Whether a wait of this CTA has given up, agreed on by the warp.
__device__ __forceinline__ bool stopped(volatile int* abort) { return __any_sync(0xffffffffu, *abort != 0); }

__device__ __forceinline__ int64_t pair_scan(int64_t v, int64_t* warp_sum) {   // inclusive, over the CTA
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) v += warp_sum[w];
  return v;
}

// Bits [at, at + 32) of a row of words, bits outside it 0.
__device__ __forceinline__ uint32_t bits_at(const int32_t* words, int n_words, int64_t at) {
  const int64_t w = at >> 5;
  const uint32_t lo = w >= 0 && w < n_words ? __ldg(words + w) : 0u;
  const uint32_t hi = w + 1 >= 0 && w + 1 < n_words ? __ldg(words + w + 1) : 0u;
  return __funnelshift_r(lo, hi, static_cast<uint32_t>(at) & 31u);
}

// TREE: a token sees every key in front of its request's new ones, and of those the ones in its mask: two words of it for a lane's
// 32 keys, read while S of the block is on its way, in the one to three blocks of a tile that hold new keys.  The mask costs
// nothing that could be measured against the causal form (64 trees 421 us either way, 24 trees over 9000-32768 keys 129 us).
template <int D_QK, bool TREE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    chunk_fwd_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap half_map,
                     const __grid_constant__ CUtensorMap box_map, const __grid_constant__ CUtensorMap group_map,
                     const __grid_constant__ CUtensorMap row_map, const ChunkParams p) {
  using L = Smem<D_QK>;
  constexpr int kChunks = L::kChunks;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* s_q = smem;
  uint8_t* s_kv = smem + L::kQBytes;
  uint8_t* s_p = smem + L::kP;
  Control& c = *reinterpret_cast<Control*>(smem + L::kControl);

  cudaTriggerProgrammaticLaunchCompletion();   // the joining kernel may come up; it waits for this one's end
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int64_t first_pair = TREE ? pair / kTreeGroup * kTreeGroup : pair;   // of those that share a range
  volatile int* abort = &c.abort_flag;

  if (tid == 0) {
    c.abort_flag = 0;
    for (int i = 0; i < kRing; ++i) {
      mbar_init(smem_u32(&c.ring_full[i]), 1);
      mbar_init(smem_u32(&c.ring_empty[i]), rank == 0 ? 8 : 6);   // two loaders, four softmax warps, two issuers
    }
    for (int i = 0; i < kGens; ++i) {
      mbar_init(smem_u32(&c.k_full[i]), 1);
      mbar_init(smem_u32(&c.x_full[i]), 1);
      mbar_init(smem_u32(&c.s_full[i]), 1);
      mbar_init(smem_u32(&c.pv_done[i]), 1);
    }
    mbar_init(smem_u32(&c.p_full), 8);     // the softmax warps of both CTAs
    mbar_init(smem_u32(&c.o_free), 8);
    mbar_init(smem_u32(&c.q_full), 1);
    fence_mbar_init();
  }
  if (warp == 3) {
    tmem_alloc_pair(smem_u32(&c.tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  if (tid == 32) {
    prefetch_map(&q_map);
    prefetch_map(&half_map);
    prefetch_map(&box_map);
    prefetch_map(&group_map);
    prefetch_map(&row_map);
  }
  tc_fence_before();
  __syncwarp();
  cluster_arrive();   // barriers and tensor memory of this CTA are ready
  // The scheduler finds this pair's range of the axis.  With 32 requests at most its warp does so alone;
  // with more, the CTA's threads sum the requests' lengths and find the request in which the range
  // starts (from the same sums when each thread has one request at most).
  RangeScan& scan = *reinterpret_cast<RangeScan*>(s_p);
  if (p.n_req > 32) {
    int64_t mine = 0;
    for (int64_t b = tid; b < p.n_req; b += kPairThreads) mine += axis_of(p, request(p, b));
    if (tid == 0) scan.req = -1;
    const int64_t upto = pair_scan(mine, scan.warp_sum);
    if (tid == kPairThreads - 1) scan.total = scan.run = upto;
    __syncthreads();
    const int64_t v0 = first_pair * range_of(scan.total, pairs);
    if (p.n_req <= kPairThreads) {
      if (upto - mine <= v0 && v0 < upto) {
        scan.req = tid;
        scan.start = upto - mine;
      }
      __syncthreads();
    } else if (v0 < scan.total) {
      int64_t run = 0;
      for (int64_t b0 = 0; b0 < p.n_req && run <= v0; b0 += kPairThreads) {
        const int64_t cost = b0 + tid < p.n_req ? axis_of(p, request(p, b0 + tid)) : 0;
        const int64_t end = run + pair_scan(cost, scan.warp_sum);
        if (end - cost <= v0 && v0 < end) {
          scan.req = b0 + tid;
          scan.start = end - cost;
        }
        if (tid == kPairThreads - 1) scan.run = end;
        __syncthreads();
        run = scan.run;
        __syncthreads();
      }
    }
  }
  __syncwarp();
  cluster_wait();     // and those of the other CTA
  tc_fence_after();
  const uint32_t tmem = c.tmem_slot;

  if (warp >= 4 && warp < 8) {
    // ============================================================ softmax and rescaling
    const int t = tid - 128;                       // TMEM lane
    const int row = (t & 63) + 64 * static_cast<int>(rank);
    const int half = t >> 6;                       // keys and value columns of this lane
    const uint32_t lanes = tmem + (static_cast<uint32_t>(t & 96) << 16);
    const uint32_t bar_id = 1 + ((t >> 5) & 1);    // the two warps that share rows
    const float scale2 = p.sm_scale * kLog2e;
    const uint32_t p_full = map_to_rank(smem_u32(&c.p_full), 0);
    uint8_t* p_row = s_p + (t & 63) * 128;
    const int sw = t & 7;
    float m = -INFINITY, top = -INFINITY, l = 0.f;   // exponent offset (log2 units), max of q.k, sum
    int b = 0;
    uint32_t tile = 0;
    int limit = 0;                                   // first key position this row does not see
    // The two warps that share rows meet at one barrier in every round, the last one included; all four meet at
    // a tile's end, or else behind the loop.  So all leave in the same tile, also when a wait gave up.
    bool agreed = false;
    for (;; ++b) {
      const BlockDesc& d = c.ring[b % kRing];
      const int g = b % kGens;
      wait_on(&c.ring_full[b % kRing], (b / kRing) & 1, abort);
      __syncwarp();
      const uint32_t flags = __shfl_sync(0xffffffffu, d.flags, 0);
      if (flags & kEnd) {
        named_bar_or(bar_id, 64, *abort != 0);
        break;
      }
      const int n_rows = d.n_rows, part = d.part;
      const int64_t q_row = d.q_row;
      const uint32_t key_mask = d.mask[half];
      const int key0 = d.key0 + 32 * half;
      if (flags & kFirst) {
        const int64_t seen = TREE ? d.pos0 : p.causal ? static_cast<int64_t>(d.pos0) + (p.groups == 1 ? row / p.h_q : 0) + 1 : d.key_end;
        limit = row < n_rows ? static_cast<int>(min(max(seen, static_cast<int64_t>(0)), static_cast<int64_t>(d.key_end))) : 0;
        m = top = -INFINITY;
        l = 0.f;
      }
      const int first_new = d.pos0;                  // TREE: position of the request's first new token
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.ring_empty[b % kRing]));
      const int n_seen = limit - key0;
      uint32_t mask = n_seen >= 32 ? key_mask : n_seen <= 0 ? 0u : key_mask & ((1u << n_seen) - 1u);
      if constexpr (TREE) {
        if (n_seen < 32 && row < n_rows)
          mask |= key_mask & bits_at(p.tree_mask + static_cast<int64_t>(static_cast<uint32_t>(q_row + row) / static_cast<uint32_t>(p.h_q)) * p.mask_words,
                                     p.mask_words, static_cast<int64_t>(key0) - first_new);
      }

      wait_on(&c.s_full[g], (b / kGens) & 1, abort);
      __syncwarp();
      tc_fence_after();
      uint32_t raw[32];
      tmem_ld32(lanes + kTmemS + 32 * g, raw);
      tmem_ld_wait();
      float s[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(raw[i]);
      if (mask != 0xffffffffu) {
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i] = (mask >> i) & 1u ? s[i] : -INFINITY;
      }
      float bm = s[0];
#pragma unroll
      for (int i = 1; i < 32; ++i) bm = fmaxf(bm, s[i]);
      c.ex[b & 1][t] = bm;
      if (named_bar_or(bar_id, 64, *abort != 0)) break;
      bm = fmaxf(bm, c.ex[b & 1][t ^ 64]);
      top = fmaxf(top, bm);
      float alpha = 1.f;
      if (bm * scale2 > m + kRescaleLog2) {
        alpha = fast_exp2(m - bm * scale2);   // 0 when m was -inf
        m = bm * scale2;
      }
      const float neg_m = m == -INFINITY ? 0.f : -m;
      float sum = 0.f;
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float e0 = fast_exp2(fmaf(s[2 * i], scale2, neg_m));
        const float e1 = fast_exp2(fmaf(s[2 * i + 1], scale2, neg_m));
        sum += e0 + e1;
        // The weights of V are rounded to bf16, since the tensor unit takes both operands in one type and V is bf16:
        // 2^-8 of a weight at most, which a sum over many keys averages (the output's whole error is 1.7e-3 to 2.1e-3
        // of its size against 1.7e-3 for its own rounding alone).  Two products, of a weight's high and low parts, would
        // avoid it at 1.4 times the block's time on the tensor unit.  The sum, and with it lse, takes the unrounded ones.
        w[i] = pack_bf16x2(e0, e1);
      }
      l = fmaf(l, alpha, sum);
      // PV of the block before has read the P tile and is done with O
      if (b > 0) wait_on(&c.pv_done[(b - 1) % kGens], ((b - 1) / kGens) & 1, abort);
      if (!(flags & kFirst) && __any_sync(0xffffffffu, alpha != 1.f)) {
        tc_fence_after();
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          uint32_t o[32];
          tmem_ld32(lanes + 32 * i, o);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
          tmem_st32(lanes + 32 * i, o);
        }
        tmem_st_wait();
      }
      // P tile: 64 rows of 64 keys, 128-byte swizzle
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(p_row + (((4 * half + i) ^ sw) << 4)) =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(p_full);

      if (flags & kLast) {
        // l of both key halves; the second barrier keeps the next block's maxima off these slots
        c.ex[(b + 1) & 1][t] = l;
        named_bar_sync(bar_id, 64);
        l += c.ex[(b + 1) & 1][t ^ 64];
        if (named_bar_or(kAgreeBar, 128, *abort != 0)) {
          agreed = true;
          break;
        }
        // Without a key l is exactly 0; with one it is about 1 at least, the term of the row's largest score, or
        // NaN, or 0 with m = +inf where a finite score leaves fp32's range once scaled: lse = m + log2 0 is NaN then, and
        // O = 0 / 0.  fmaxf passes over NaN scores, so the maximum takes its NaN from the sum.
        const bool empty = l == 0.f && m < INFINITY;
        const float largest = empty ? -INFINITY : l == l ? top * p.sm_scale : l;
        const bool live = row < n_rows;
        float inv = 1.f;
        if (part < 0) {
          const int64_t r = q_row + row;
          float den = l;
          if (p.attn_sink && live) den += exp2f(fmaf(__ldg(p.attn_sink + r % p.h_q), kLog2e, -m));
          inv = empty ? 0.f : 1.f / den;
          if (live && half == 0) {
            p.lse[r] = empty ? INFINITY : (m + log2f(l)) * kLn2;
            p.max_logits[r] = largest;
          }
        } else if (live && half == 0) {
          float* st = p.part_stats + part * 3 * 128 + row;
          st[0] = empty ? -INFINITY : m;
          st[128] = l;
          st[256] = largest;
        }
        // The epilogue warps take it from here.  Two slots of factors are enough: this group's next tile but one
        // comes behind PV of its next tile, which waits until they have read O of this one.
        if (half == 0) c.inv[tile & 1][t] = inv;
        if (t == 0) {
          auto& done = c.done[tile % kTileBars];
          done.q_row = static_cast<int32_t>(q_row);
          done.n_rows = n_rows;
          done.part = part;
          done.last = b;
        }
        named_bar_arrive(kTileBar + tile % kTileBars, 256);
        ++tile;
      }
    }
    if (!agreed) named_bar_or(kAgreeBar, 128, true);
    if (b > 0) wait_on(&c.pv_done[(b - 1) % kGens], ((b - 1) / kGens) & 1, abort);
    if (t == 0) c.done[tile % kTileBars].last = -1;
    __syncwarp();
    named_bar_arrive(kTileBar + tile % kTileBars, 256);
  } else if (warp >= 8 && warp < 12) {
    // ============================================================ epilogue
    // Warps of its own, so that the softmax of the next tile need not wait (9500 cycles between two tiles
    // without, 3500 with them), asleep on a named barrier: waiting on an mbarrier, the four warps took so many issue
    // slots from the softmax warps next to them that all calls ran 1.6 times as long.
    const int t = tid - 256, row = (t & 63) + 64 * static_cast<int>(rank), half = t >> 6;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(t & 96) << 16);
    const uint32_t o_free = map_to_rank(smem_u32(&c.o_free), 0);
    for (uint32_t tile = 0;; ++tile) {
      const auto& d = c.done[tile % kTileBars];
      named_bar_sync(kTileBar + tile % kTileBars, 256);   // the softmax warps arrive for each tile and for the end
      const int last = d.last, n_rows = d.n_rows, part = d.part;
      if (last < 0) break;
      const int64_t q_row = d.q_row;
      const float inv = c.inv[tile & 1][t & 63];
      wait_on(&c.pv_done[last % kGens], (last / kGens) & 1, abort);
      __syncwarp();
      tc_fence_after();
      // A lane holds a row's 256 values; stored as they are, each store instruction would touch 32 rows.
      // Four lanes exchange their rows' pieces of 64 bytes first, so that each store covers 64 bytes of
      // eight rows.  A part of a tile goes to the workspace as it lies here: four columns of all rows
      // together.
      const int row4 = row - (lane & 3);
      __nv_bfloat16* out = p.out + (q_row + row4) * kDv + 256 * half + 8 * (lane & 3);
      float4* po = reinterpret_cast<float4*>(p.part_o) + (static_cast<int64_t>(part) * 128 + 64 * half) * p.row_cap + row;
      auto put = [&](const uint32_t(&o)[32], int i) {   // columns 32 i .. 32 i + 31
        if (part < 0) {
          uint32_t v[4][4];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float a = __uint_as_float(o[2 * j]), e = __uint_as_float(o[2 * j + 1]);
            v[j >> 2][j & 3] = inv == 0.f ? 0u : pack_bf16x2(a * inv, e * inv);
          }
          transpose_4x4(v, lane);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (row4 + x < n_rows)
              *reinterpret_cast<uint4*>(out + x * kDv + 32 * i) = make_uint4(v[x][0], v[x][1], v[x][2], v[x][3]);
        } else if (row < n_rows) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            po[(8 * i + j) * p.row_cap] = make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]),
                                                      __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]));
        }
        __syncwarp();
      };
#pragma unroll 1
      for (int i = 0; i < 8; i += 2) {
        uint32_t o0[32], o1[32];
        tmem_ld32(lanes + 32 * i, o0);
        tmem_ld32(lanes + 32 * i + 32, o1);
        tmem_ld_wait();
        if (i == 6) {   // O has been read: the next tile's first PV may overwrite it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_pair(o_free);
        }
        put(o0, i);
        put(o1, i + 1);
      }
    }
  } else if (warp == 0) {
    // ============================================================ scheduler
    int b = 0;
    bool stop = false;
    auto acquire = [&] {
      if (b >= kRing) wait_on(&c.ring_empty[b % kRing], ((b / kRing) - 1) & 1, abort);
      stop = stopped(abort);
    };
    auto publish = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.ring_full[b % kRing]));
      ++b;
    };
    int4 join = make_int4(0, 0, -1, 0);
    int64_t join_end = 0, join_start = 0;
    const bool few = p.n_req <= 32;
    Request mine{};                              // of request `window` + lane
    int64_t window = 0;
    int64_t total, start, first_req;             // start: the request's position on the axis
    int64_t range, v0;
    if (few) {
      int64_t cost = 0;
      if (lane < p.n_req) {
        mine = request(p, lane);
        cost = axis_of(p, mine);
      }
      int64_t end = cost;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += u;
      }
      total = __shfl_sync(0xffffffffu, end, 31);
      range = range_of(total, pairs);
      v0 = first_pair * range;
      const uint32_t hit = __ballot_sync(0xffffffffu, end - cost <= v0 && v0 < end);
      first_req = __ffs(hit) - 1;                // -1: the range lies behind the axis' end
      start = __shfl_sync(0xffffffffu, end - cost, hit ? __ffs(hit) - 1 : 0);
    } else {
      total = scan.total;
      range = range_of(total, pairs);
      v0 = first_pair * range;
      first_req = scan.req;
      start = scan.start;
    }
    const int64_t members = TREE ? min(static_cast<int64_t>(kTreeGroup), pairs - first_pair) : 1;
    const int64_t v1 = v0 + members * range;
    // TREE: the pairs that share a range take its tiles in turn, each tile to the least loaded one, as long as it fits; what is then
    // left of the range goes to them in pieces, in order: [a, e) to this one.  A tile longer than a pair's share is cut as in
    // the causal form, and there are no more cuts than there.
    int64_t load[kTreeGroup], a = v0, e = v1;
#pragma unroll
    for (int g = 0; g < kTreeGroup; ++g) load[g] = g < members ? 0 : range;
    bool pieces = !TREE;
    bool more = v0 < total && first_req >= 0;
    // The tree form has several tiles on one request's keys, one after the other, and all requests' keys together may be more
    // than the L2 holds.  So four neighbouring pairs share a range and take its tiles in turn (above), and each walks one tile's
    // keys forward and its next one's backward, which begins with what is still there.  64 trees of 6-16 nodes, 128 heads,
    // 1024-4096 keys: 1.6 GB from DRAM without the sharing, 0.6 with it; alone and forward 421 us, alone in turns 406, by four in
    // turns 399 (over seconds, at the power limit: 474, 454, 428); 64 of 19 nodes over 2560 keys 635, 613, 592 (731, 690, 643).
    // Keys that fit the L2 gain nothing (16 trees of 19 nodes over 10240: 565, 560, 565).  By two pairs 398 and 594 us, but 48
    // trees of 8 nodes over 8192 keys 629 instead of 601; by eight 432: too many ask for the same rows at once.
    bool back = true;
    if (!few) window = -32;                      // loaded below
    for (int64_t req = first_req; more && req < p.n_req && start < total && !stop; ++req) {
      if (req >= window + 32 || window < 0) {
        window = req;
        mine = Request{};
        if (window + lane < p.n_req) mine = request(p, window + lane);
      }
      // the next request with tokens
      const uint32_t live = __ballot_sync(0xffffffffu, mine.n_q > 0) >> (req - window);
      if (live == 0u) {
        req = window + 31;
        continue;
      }
      req += __ffs(live) - 1;
      const int from = static_cast<int>(req - window);
      Request r;
      r.q0 = __shfl_sync(0xffffffffu, mine.q0, from);
      r.n_q = __shfl_sync(0xffffffffu, mine.n_q, from);
      r.n_k = __shfl_sync(0xffffffffu, mine.n_k, from);
      r.keys = __shfl_sync(0xffffffffu, mine.keys, from);
      const int64_t n_tiles = token_tiles(p, r);
      const int64_t before = r.n_k - r.n_q;      // position of the request's first new token
      int64_t k = 0, s = start;                  // token tile, its position on the axis
      if (start < v0) {   // the range starts inside this request: last token tile that begins at or before v0
        int64_t lo = 0, hi = n_tiles;
        while (hi - lo > 1) {
          const int64_t mid = (lo + hi) >> 1;
          if (axis_of(p, r, mid, n_tiles) <= v0 - start) lo = mid;
          else hi = mid;
        }
        k = lo;
        s = start + axis_of(p, r, k, n_tiles);
      }
      for (; k < n_tiles && more && !stop; ++k) {
        const int64_t tok = k * p.tokens_per_tile, last = min(r.n_q, tok + p.tokens_per_tile);
        const int64_t size = kTileCost + (p.causal ? max(before, static_cast<int64_t>(0)) + last : r.n_k);
        const int64_t key_end = p.causal ? min(max(before + last, static_cast<int64_t>(0)), r.keys) : r.keys;
        const int64_t n_blocks = max((key_end + kKeys - 1) / kKeys, static_cast<int64_t>(1));
        for (int grp = 0; grp < p.groups && more && !stop; ++grp, s += size) {
          if (s >= e) {
            more = false;
            break;
          }
          if (!pieces) {
            if (s + size <= v0) continue;        // another group of heads of the token in which the range starts
            const int64_t begin = max(s, v0), len = s + size - begin;
            int to = 0;
            int64_t least = load[0];
#pragma unroll
            for (int g = 1; g < kTreeGroup; ++g)
              if (load[g] < least) {
                least = load[g];
                to = g;
              }
            if (s + size <= v1 && least + len <= range) {
#pragma unroll
              for (int g = 0; g < kTreeGroup; ++g) load[g] += g == to ? len : 0;
              if (first_pair + to != pair) continue;
            } else {
              pieces = true;
              e = begin;
#pragma unroll
              for (int g = 0; g < kTreeGroup; ++g)
                if (first_pair + g <= pair) {
                  a = e;
                  e += range - load[g];
                }
              if (s >= e) {
                more = false;
                break;
              }
            }
          }
          const int64_t j0 = s >= a ? 0 : (a - s + kKeys - 1) / kKeys;
          const int64_t j1 = min(n_blocks, (e - s + kKeys - 1) / kKeys);
          if (j0 >= j1) continue;
          const int64_t q_row = (r.q0 + tok) * p.h_q + (p.groups > 1 ? kTileRows * grp : 0);
          const int n_rows = p.groups > 1 ? min(kTileRows, p.h_q - kTileRows * grp) : static_cast<int>(last - tok) * p.h_q;
          int part = -1;
          if (j0 > 0) part = static_cast<int>(2 * pair);
          else if (j1 < n_blocks) {
            part = static_cast<int>(2 * pair + 1);
            join = make_int4(static_cast<int>(q_row), n_rows, 0, 0);
            join_end = s + kKeys * (n_blocks - 1);   // the tile's last block: in the range of the last pair
            join_start = s;
          }
          back = TREE && !back;
          for (int64_t i = j0; i < j1 && !stop; ++i) {
            const int64_t j = back ? j0 + j1 - 1 - i : i;
            int32_t pool_row[2];
            uint32_t mask[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int64_t pos = kKeys * j + 32 * x + lane;
              int64_t at_row = -1;
              if (pos < key_end) {   // so the column is below max_blocks
                const int col = static_cast<int>(pos) / p.page_block;
                const int64_t page = __ldg(p.block_table + req * p.max_blocks + col);
                at_row = page * p.page_block + (static_cast<int>(pos) - col * p.page_block);
                if (page < 0 || at_row >= p.pool_rows) at_row = -1;
              }
              pool_row[x] = static_cast<int32_t>(at_row);
              mask[x] = __ballot_sync(0xffffffffu, at_row >= 0);
            }
            acquire();
            BlockDesc& d = c.ring[b % kRing];
            d.rows[lane] = pool_row[0];
            d.rows[32 + lane] = pool_row[1];
            if (lane == 0) {
              d.mask[0] = mask[0];
              d.mask[1] = mask[1];
              d.flags = (i == j0 ? kFirst : 0u) | (i == j1 - 1 ? kLast : 0u);
              d.key0 = static_cast<int32_t>(kKeys * j);
              d.q_row = static_cast<int32_t>(q_row);
              d.n_rows = n_rows;
              d.pos0 = static_cast<int32_t>(TREE ? before : before + tok);
              d.key_end = static_cast<int32_t>(key_end);
              d.part = part;
            }
            publish();
          }
        }
      }
      start = s;
    }
    if (join.z == 0) {   // the pair that has the cut tile's last block, and (w) which ones in between have none of it
      join.z = static_cast<int>(join_end / range);
      if (TREE) {
        if (join_end < e) join.z = static_cast<int>(pair);
        int64_t begin = e;
#pragma unroll
        for (int g = 1; g < kTreeGroup; ++g)
          if (first_pair + g > pair && begin <= join_end) {
            const int64_t end = begin + range - load[g];
            if (join_end < v1) join.z = static_cast<int>(first_pair + g);
            if ((begin - join_start + kKeys - 1) / kKeys == (end - join_start + kKeys - 1) / kKeys) join.w |= 1 << (first_pair + g - pair);
            begin = end;
          }
      }
    }
    acquire();
    if (lane == 0) {
      c.ring[b % kRing].flags = kEnd;
      if (rank == 0) p.joins[pair] = join;
    }
    publish();
  } else if (warp == 1 || warp == 2) {
    // ============================================================ key loads
    // Warp 1: all columns of the CTA's own 32 keys.  Warp 2: the CTA's value columns of the other CTA's 32
    // keys, in place of the foreign half, and each tile's Q, as soon as S of the tile before is done.  One
    // elected thread issues the loads: issued from several lanes, each costs the warp a turn (a chunk of
    // 2048 tokens took 2.95 ms instead of 2.85).
    const bool foreign = warp == 2;
    const uint32_t k_full = map_to_rank(smem_u32(&c.k_full[0]), 0), x_full = map_to_rank(smem_u32(&c.x_full[0]), 0);
    const uint32_t q_full = map_to_rank(smem_u32(&c.q_full), 0);
    const int which = static_cast<int>(foreign ? 1 - rank : rank);   // the half of the block's keys that this warp loads
    // n_chunks 64-column chunks from chunk0 on, 4096 bytes each.  32 keys that all count go by tiled loads,
    // four chunks at once where they lie in one page.  Otherwise groups of eight rows go by tiled loads where
    // all eight keys count, or none (a group behind the pool's end reads as zeros), and mixed groups row by
    // row (row -1 reads as zeros).
    auto load = [&](const BlockDesc& d, int chunk0, int n_chunks, uint32_t dst, uint32_t bar) {
      const uint32_t mask = d.mask[which];
      const int32_t* rows = d.rows + 32 * which;
      if (p.box == 32 && mask == 0xffffffffu && n_chunks == 4) {
        tma_load_3d_pair(dst, &half_map, 0, rows[0], chunk0, bar);
      } else if (p.box > 0 && mask == 0xffffffffu) {
        for (int k0 = 0; k0 < 32; k0 += p.box)
          for (int ch = 0; ch < n_chunks; ++ch)
            tma_load_2d_pair(dst + ch * 4096 + k0 * 128, &box_map, 64 * (chunk0 + ch), rows[k0], bar);
      } else {
        for (int k0 = 0; k0 < 32; k0 += 8, rows += 8, dst += 1024) {
          const uint32_t group = (mask >> k0) & 0xffu;
          if (p.box > 0 && (group == 0u || group == 0xffu)) {
            const int row = group ? rows[0] : p.pool_end;
            for (int ch = 0; ch < n_chunks; ++ch)
              tma_load_2d_pair(dst + ch * 4096, &group_map, 64 * (chunk0 + ch), row, bar);
          } else {
            for (int x = 0; x < 8; x += 4) {
              const int4 rr = *reinterpret_cast<const int4*>(rows + x);
              for (int ch = 0; ch < n_chunks; ++ch)
                tma_gather4_pair(dst + ch * 4096 + x * 128, &row_map, 64 * (chunk0 + ch), rr.x, rr.y, rr.z, rr.w, bar);
            }
          }
        }
      }
    };
    auto load_q = [&](const BlockDesc& d) {
      if (elect_one()) {
        if (rank == 0) mbar_arrive_expect_tx(smem_u32(&c.q_full), 2 * L::kQBytes);
        const int q_row = d.q_row + 64 * static_cast<int>(rank);
        for (int ch = 0; ch < kChunks; ++ch) tma_load_2d_pair(smem_u32(s_q + ch * 8192), &q_map, 64 * ch, q_row, q_full);
      }
      __syncwarp();
    };
    for (int b = 0;; ++b) {
      const BlockDesc& d = c.ring[b % kRing];
      const int g = b % kGens;
      wait_on(&c.ring_full[b % kRing], (b / kRing) & 1, abort);
      if (stopped(abort)) break;
      const uint32_t flags = d.flags;
      if (flags & kEnd) break;
      const uint32_t gen = smem_u32(s_kv) + g * L::kGenBytes;
      if (foreign) {
        if (b == 0) load_q(d);
        wait_on(&c.s_full[g], (b / kGens) & 1, abort);   // S has read the foreign half, and at a tile's end Q
        if (stopped(abort)) break;
        if (flags & kLast) {
          const BlockDesc& next = c.ring[(b + 1) % kRing];
          wait_on(&c.ring_full[(b + 1) % kRing], ((b + 1) / kRing) & 1, abort);
          if (stopped(abort)) break;
          if (!(next.flags & kEnd)) load_q(next);
        }
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(smem_u32(&c.x_full[g]), 2 * kHalfBytes);
          load(d, 4 * static_cast<int>(rank), 4, gen + (1 - rank) * kHalfBytes, x_full + 8 * g);
        }
      } else {
        if (b >= kGens) wait_on(&c.pv_done[g], ((b / kGens) - 1) & 1, abort);
        if (stopped(abort)) break;
        if (elect_one()) {
          const uint32_t bar = k_full + 8 * g;
          if (rank == 0) mbar_arrive_expect_tx(smem_u32(&c.k_full[g]), 2 * L::kGenBytes);
          if constexpr (kChunks > 8) load(d, 8, 1, gen + 2 * kHalfBytes, bar);
          load(d, 0, 4, gen, bar);
          load(d, 4, 4, gen + kHalfBytes, bar);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.ring_empty[b % kRing]));
    }
  } else if (warp == 3 && rank == 0) {
    // ============================================================ S issuer
    if (elect_one()) {
      constexpr uint32_t idesc = make_idesc_bf16(kTileRows, kKeys, false, false);
      const uint64_t qd = make_sdesc_sw128(smem_u32(s_q), 16, 1024);
      int64_t tiles = 0;
      for (int b = 0; !*abort; ++b) {
        const int g = b % kGens;
        wait_on(&c.ring_full[b % kRing], (b / kRing) & 1, abort);
        const uint32_t flags = c.ring[b % kRing].flags;
        mbar_arrive(smem_u32(&c.ring_empty[b % kRing]));
        if (flags & kEnd) break;
        if (flags & kFirst) wait_on(&c.q_full, tiles++ & 1, abort);
        // the keys have landed; their loads waited for PV of block b - 4, so S buffer g has been read
        wait_on(&c.k_full[g], (b / kGens) & 1, abort);
        tc_fence_after();
        const uint64_t kd = make_sdesc_sw128(smem_u32(s_kv) + g * L::kGenBytes, 16, 1024);
#pragma unroll
        for (int ks = 0; ks < D_QK / 16; ++ks)
          umma_ss_pair(tmem + kTmemS + 32 * g, qd + (((ks >> 2) * 8192 + (ks & 3) * 32) >> 4),
                       kd + (((ks >> 2) * 4096 + (ks & 3) * 32) >> 4), idesc, ks > 0 ? 1u : 0u);
        umma_commit_pair(smem_u32(&c.s_full[g]));
      }
    }
    __syncwarp();
  } else if (warp == 12 && rank == 0) {
    // ============================================================ PV issuer
    if (elect_one()) {
      constexpr uint32_t idesc = make_idesc_bf16(kTileRows, 256, false, true);
      const uint64_t pd = make_sdesc_sw128(smem_u32(s_p), 16, 1024);
      int64_t tiles = 0;
      for (int b = 0; !*abort; ++b) {
        const int g = b % kGens;
        wait_on(&c.ring_full[b % kRing], (b / kRing) & 1, abort);
        const uint32_t flags = c.ring[b % kRing].flags;
        mbar_arrive(smem_u32(&c.ring_empty[b % kRing]));
        if (flags & kEnd) break;
        const bool first = (flags & kFirst) != 0;
        if (first) {   // the tile before has been read out of O
          if (tiles > 0) wait_on_pair(&c.o_free, (tiles - 1) & 1, abort);
          ++tiles;
        }
        wait_on(&c.x_full[g], (b / kGens) & 1, abort);
        wait_on_pair(&c.p_full, b & 1, abort);
        tc_fence_after();
        // keys 0-31 in D0, 32-63 in D1, in both CTAs (own and foreign, or foreign and own)
        const uint64_t vd = make_sdesc_sw128(smem_u32(s_kv) + g * L::kGenBytes, 4096, 1024);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int ks = 0; ks < kKeys / 16; ++ks)
            umma_ss_pair(tmem + 128 * n, pd + ((ks * 32) >> 4),
                         vd + (((ks >> 1) * kHalfBytes + n * 8192 + (ks & 1) * 2048) >> 4), idesc,
                         (!first || ks > 0) ? 1u : 0u);
        umma_commit_pair(smem_u32(&c.pv_done[g]));
      }
      // the only arrivals of the other CTA that nothing else waits for: it may not outlive them
      if (tiles > 0) wait_on_pair(&c.o_free, (tiles - 1) & 1, abort);
    }
    __syncwarp();
  }

  // ---- Every copy and product has been waited for (each tile's epilogue follows its last PV) unless a wait
  // gave up, in either CTA; then what is still in flight gets time to land before the CTAs leave.
  __syncwarp();
  if (*abort && lane == 0) store_pair(map_to_rank(smem_u32(&c.abort_flag), 1 - rank), 1);
  __syncwarp();
  tc_fence_before();
  if (*abort) cluster_arrive();
  else cluster_arrive_relaxed();   // nothing to publish: the kernel's end makes its results visible
  cluster_wait();
  if (*abort) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 5000000ull) {
    }
    __syncwarp();
  }
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------------ joining cut tiles
// A tile cut over pairs w .. w1 left its parts in slots 2w + 1, 2(w+1), .., 2 w1.  With M = max m_i:
//   l = sum 2^(m_i - M) l_i,   O = sum 2^(m_i - M) O_i / (l + [sink] 2^(sink log2 e - M)).
// A CTA takes 32 rows and 64 columns, a lane a row: the parts are read as they were written, 16 bytes of 32
// rows at a time, with the loads of three parts in flight, and the output leaves through shared memory in
// whole row pieces.  Latency bounds it: a round trip to parts that other SMs have just written takes 1.3 us.
// The kernel adds 5 us to a call with twelve parts, 8 us to 256 requests (70 cut tiles, 36 MB of parts).
constexpr int kJoinRows = 32;
constexpr int kJoinWarps = 8;                 // two column quads each
constexpr int kJoinParts = 3;

__global__ void __launch_bounds__(32 * kJoinWarps) chunk_join_kernel(const ChunkParams p) {
  __shared__ __align__(16) uint2 tile[kJoinRows][17];   // four columns each; padded against bank conflicts
  const int w = blockIdx.x;
  cudaGridDependencySynchronize();
  const int4 join = p.joins[w];
  const int row0 = blockIdx.y * kJoinRows;
  if (join.z < 0 || row0 >= join.y) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = min(row0 + lane, join.y - 1);         // lanes behind the last row repeat it
  const int64_t r = static_cast<int64_t>(join.x) + row;
  const float sink2 = p.attn_sink ? __ldg(p.attn_sink + r % p.h_q) * kLog2e : -INFINITY;
  const float* stats = p.part_stats + row;
  const float4* part = reinterpret_cast<const float4*>(p.part_o) + (16 * blockIdx.z + 2 * warp) * p.row_cap + row;
  float M = -INFINITY, top = -INFINITY, l = 0.f;
  float4 acc[2] = {};
  for (int i0 = w; i0 <= join.z; i0 += kJoinParts) {
    float m[kJoinParts], li[kJoinParts], ti[kJoinParts];
    float4 o[kJoinParts][2];
#pragma unroll
    for (int u = 0; u < kJoinParts; ++u) {
      const int i = min(i0 + u, join.z), slot = i == w ? 2 * w + 1 : 2 * i;
      const float* st = stats + slot * 3 * 128;
      const bool none = i - w < 32 && (join.w >> (i - w)) & 1;
      m[u] = none ? -INFINITY : st[0];
      li[u] = none ? 0.f : st[128];
      ti[u] = none ? -INFINITY : st[256];
#pragma unroll
      for (int x = 0; x < 2; ++x)
        o[u][x] = none ? float4{} : part[(static_cast<int64_t>(slot) * 128 + x) * p.row_cap];
    }
    float now = M;
#pragma unroll
    for (int u = 0; u < kJoinParts; ++u)
      if (i0 + u <= join.z) now = fmaxf(now, m[u]);
    const float base = now > -INFINITY ? now : 0.f, keep = exp2f(M - base);
    M = now;
    l *= keep;
#pragma unroll
    for (int x = 0; x < 2; ++x) acc[x] = make_float4(acc[x].x * keep, acc[x].y * keep, acc[x].z * keep, acc[x].w * keep);
#pragma unroll
    for (int u = 0; u < kJoinParts; ++u) {
      if (i0 + u > join.z) break;
      const float a = exp2f(m[u] - base);
      l = fmaf(a, li[u], l);
      top = fmaxf(top, ti[u]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        acc[x].x = fmaf(a, o[u][x].x, acc[x].x);
        acc[x].y = fmaf(a, o[u][x].y, acc[x].y);
        acc[x].z = fmaf(a, o[u][x].z, acc[x].z);
        acc[x].w = fmaf(a, o[u][x].w, acc[x].w);
      }
    }
  }
  const bool empty = l == 0.f;   // a part's NaN reaches the sum of all parts
  const float den = p.attn_sink && !empty ? l + exp2f(sink2 - M) : l;
  const float inv = empty ? 0.f : 1.f / den;
#pragma unroll
  for (int x = 0; x < 2; ++x)
    tile[lane][2 * warp + x] = empty ? make_uint2(0u, 0u)
                                     : make_uint2(pack_bf16x2(acc[x].x * inv, acc[x].y * inv),
                                                  pack_bf16x2(acc[x].z * inv, acc[x].w * inv));
  if (row0 + lane < join.y && warp == 0 && blockIdx.z == 0) {
    p.lse[r] = empty ? INFINITY : (M + log2f(l)) * kLn2;
    p.max_logits[r] = l == l ? top : l;   // -inf for an empty row
  }
  __syncthreads();
  for (int k = warp; k < kJoinRows && row0 + k < join.y; k += kJoinWarps)
    if (lane < 16) reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(join.x) + row0 + k) * kDv + 64 * blockIdx.z)[lane] = tile[k][lane];
}

// ------------------------------------------------------------------------ wait self-test
// Both forms of the wait, on a barrier that nothing completes: each gives up after limit_ns.  A third one finds the
// flag of the first set and gives up at once, whatever its limit.
__global__ void chunk_wait_selftest_kernel(uint64_t limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag[2];
  if (threadIdx.x != 0) return;
  abort_flag[0] = abort_flag[1] = 0;
  mbar_init(smem_u32(&bar), 1);
  fence_mbar_init();
  wait_bounded<false>(&bar, 0, &abort_flag[0], limit_ns);
  wait_bounded<true>(&bar, 0, &abort_flag[1], limit_ns);
  wait_bounded<false>(&bar, 0, &abort_flag[0]);
}

// ------------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

bool encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  const auto fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t es[3] = {1, 1, 1};
  std::memset(m, 0, sizeof(*m));
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// box_rows rows of 64 columns of a row-major bf16 matrix, addressed by column and row; 128-byte swizzle.
bool map_rows(CUtensorMap* m, const void* base, int64_t rows, int cols, int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  return encode(m, base, 2, dims, strides, box);
}

// The same by (column in its chunk of 64, row, chunk): 32 rows of four chunks, chunk after chunk.
bool map_half(CUtensorMap* m, const void* base, int64_t rows, int cols) {
  const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(cols / 64)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 2, 128};
  const cuuint32_t box[3] = {64, 32, 4};
  return encode(m, base, 3, dims, strides, box);
}

struct Workspace {
  size_t stats, joins, bytes;   // offsets behind part_o
};
Workspace workspace_of(int64_t n_tok, int h_q) {
  const int64_t cap = n_tok * h_q < kTileRows ? n_tok * h_q : kTileRows;
  Workspace w;
  w.stats = static_cast<size_t>(2 * kMaxPairs) * cap * kDv * 4;   // multiples of 256
  w.joins = w.stats + 2 * kMaxPairs * 3 * 128 * 4;
  w.bytes = w.joins + ((kMaxPairs * sizeof(int4) + 255) & ~static_cast<size_t>(255));
  return w;
}

// SMs of the current device; 0 on an error.  Asked once per device, with the kernels' shared-memory limit set
// there at the same time.
int device_sms() {
  constexpr int kDevices = 64;
  static std::atomic<int> sms[kDevices];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
  if ((n = sms[dev].load(std::memory_order_acquire)) > 0) return n;
  constexpr auto kLimit = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if (cudaFuncSetAttribute(chunk_fwd_kernel<512, false>, kLimit, Smem<512>::kBytes) != cudaSuccess ||
      cudaFuncSetAttribute(chunk_fwd_kernel<576, false>, kLimit, Smem<576>::kBytes) != cudaSuccess ||
      cudaFuncSetAttribute(chunk_fwd_kernel<512, true>, kLimit, Smem<512>::kBytes) != cudaSuccess ||
      cudaFuncSetAttribute(chunk_fwd_kernel<576, true>, kLimit, Smem<576>::kBytes) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  sms[dev].store(n, std::memory_order_release);
  return n;
}

template <int D_QK, bool TREE>
smla_status launch(const CUtensorMap& qm, const CUtensorMap& hm, const CUtensorMap& bm, const CUtensorMap& gm,
                   const CUtensorMap& rm, const ChunkParams& p, int pairs, cudaStream_t stream) {
  chunk_fwd_kernel<D_QK, TREE><<<2 * pairs, kPairThreads, Smem<D_QK>::kBytes, stream>>>(qm, hm, bm, gm, rm, p);
  if (cudaGetLastError() != cudaSuccess) return SMLA_ERR_LAUNCH;
  // the joining kernel's CTAs come up while the first one still runs, and wait for its end
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(pairs, (p.row_cap + kJoinRows - 1) / kJoinRows, kDv / 64);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_join_kernel, p) == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

template <bool TREE>
smla_status dense_fwd(const void* q, const void* kv_pool, int64_t pool_rows, const int32_t* block_table, int max_blocks,
                      int page_block, const int32_t* cu_seqlens_q, const int32_t* seqlens_k, int64_t n_req, int causal,
                      const int32_t* tree_mask, int mask_words, const float* attn_sink, float sm_scale, int d_v, void* out,
                      float* lse, float* max_logits, int64_t n_tok, int h_q, int d_qk, void* workspace,
                      size_t workspace_bytes, smla_stream_t stream) {
  if (n_tok < 0 || n_req < 0 || n_req > INT32_MAX || h_q < 1 || h_q > 1024 || (d_qk != 512 && d_qk != 576) ||
      d_v != kDv || !(sm_scale > 0.f) || !std::isfinite(sm_scale) || n_tok > INT32_MAX / h_q ||
      (TREE && (mask_words < 1 || mask_words > 1024)))
    return SMLA_ERR_BAD_SHAPE;
  if (n_tok == 0 || n_req == 0) return SMLA_OK;
  if (pool_rows < 1 || pool_rows > INT32_MAX || max_blocks < 1 || page_block < 1 ||
      static_cast<int64_t>(max_blocks) * page_block > INT32_MAX)
    return SMLA_ERR_BAD_SHAPE;
  if (!q || !kv_pool || !block_table || !cu_seqlens_q || !seqlens_k || !out || !lse || !max_logits ||
      (TREE && !tree_mask))
    return SMLA_ERR_NULL_PTR;
  if (!aligned_to(q, 16) || !aligned_to(kv_pool, 16) || !aligned_to(out, 16) || !aligned_to(lse, 4) ||
      !aligned_to(max_logits, 4) || !aligned_to(block_table, 4) || !aligned_to(cu_seqlens_q, 4) ||
      !aligned_to(seqlens_k, 4) || !aligned_to(attn_sink, 4) || !aligned_to(tree_mask, 4))
    return SMLA_ERR_MISALIGNED;
  const Workspace ws = workspace_of(n_tok, h_q);
  if (!workspace || workspace_bytes < ws.bytes) return SMLA_ERR_WORKSPACE;
  if (!aligned_to(workspace, 256)) return SMLA_ERR_MISALIGNED;
  // tiles are finished, and parts stored, while other CTAs still read the inputs
  const size_t rows = static_cast<size_t>(n_tok) * h_q, reqs = static_cast<size_t>(n_req) * 4;
  const Span in[] = {{q, rows * d_qk * 2}, {kv_pool, static_cast<size_t>(pool_rows) * d_qk * 2},
                     {block_table, reqs * max_blocks}, {cu_seqlens_q, reqs + 4}, {seqlens_k, reqs},
                     {attn_sink, static_cast<size_t>(h_q) * 4}, {tree_mask, static_cast<size_t>(n_tok) * mask_words * 4}};
  const Span written[] = {{out, rows * kDv * 2}, {lse, rows * 4}, {max_logits, rows * 4}, {workspace, ws.bytes}};
  if (any_overlap(in, written)) return SMLA_ERR_BAD_SHAPE;
  const int sms = device_sms();
  if (sms < 2) return SMLA_ERR_LAUNCH;
  ChunkParams p{};
  p.block_table = block_table;
  p.cu_seqlens_q = cu_seqlens_q;
  p.seqlens_k = seqlens_k;
  p.attn_sink = attn_sink;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.max_logits = max_logits;
  p.part_o = static_cast<float*>(workspace);
  p.part_stats = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ws.stats);
  p.joins = reinterpret_cast<int4*>(static_cast<uint8_t*>(workspace) + ws.joins);
  p.pool_rows = pool_rows;
  p.n_req = n_req;
  p.n_tok = n_tok;
  p.sm_scale = sm_scale;
  p.h_q = h_q;
  p.max_blocks = max_blocks;
  p.page_block = page_block;
  p.causal = causal != 0;
  p.tree_mask = tree_mask;
  p.mask_words = mask_words;
  // Tiled loads take rows of one page, in groups of eight (the 128-byte swizzle's pattern): three and one for a
  // CTA's part of a block at 32 rows, against 104 gathers of four rows where the page size is not a multiple of 8.
  // 256 tokens over 1024-4096 keys: pages of 64 and 32 163-170 us, 16 185 us, 8 and 24 235 us, 100 473 us, 20 492 us, 1
  // 474 us; 4 chunks of 300-512 tokens over 2048-8192 keys, in floors: 64 and 32 1.32, 16 1.64, 8 and 24 2.25, others 5.4.
  p.box = page_block % 32 == 0 ? 32 : page_block % 16 == 0 ? 16 : page_block % 8 == 0 ? 8 : 0;
  p.pool_end = static_cast<int>(pool_rows);
  p.tokens_per_tile = h_q <= kTileRows ? kTileRows / h_q : 1;
  p.groups = h_q <= kTileRows ? 1 : (h_q + kTileRows - 1) / kTileRows;
  p.row_cap = static_cast<int>(n_tok * h_q < kTileRows ? n_tok * h_q : kTileRows);
  CUtensorMap qm, hm, bm, gm, rm;
  if (!map_rows(&qm, q, n_tok * h_q, d_qk, 64) || !map_half(&hm, kv_pool, pool_rows, d_qk) ||
      !map_rows(&bm, kv_pool, pool_rows, d_qk, p.box ? p.box : 8) || !map_rows(&gm, kv_pool, pool_rows, d_qk, 8) ||
      !map_rows(&rm, kv_pool, pool_rows, d_qk, 1))
    return SMLA_ERR_TENSOR_MAP;
  const int pairs = sms / 2 < kMaxPairs ? sms / 2 : kMaxPairs;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return d_qk == 512 ? launch<512, TREE>(qm, hm, bm, gm, rm, p, pairs, s) : launch<576, TREE>(qm, hm, bm, gm, rm, p, pairs, s);
}

}  // namespace
}  // namespace smla

using namespace smla;

extern "C" {

size_t sparse_mla_chunk_workspace_size(int64_t n_tok, int h_q) {
  if (n_tok <= 0 || h_q < 1 || h_q > 1024 || n_tok > INT32_MAX / h_q) return 0;
  return workspace_of(n_tok, h_q).bytes;
}

smla_status sparse_mla_chunk_fwd_paged(const void* q, const void* kv_pool, int64_t pool_rows,
                                       const int32_t* block_table, int max_blocks, int page_block,
                                       const int32_t* cu_seqlens_q, const int32_t* seqlens_k, int64_t n_req, int causal,
                                       const float* attn_sink, float sm_scale, int d_v, void* out, float* lse,
                                       float* max_logits, int64_t n_tok, int h_q, int d_qk, void* workspace,
                                       size_t workspace_bytes, smla_stream_t stream) {
  return dense_fwd<false>(q, kv_pool, pool_rows, block_table, max_blocks, page_block, cu_seqlens_q, seqlens_k, n_req, causal,
                          nullptr, 0, attn_sink, sm_scale, d_v, out, lse, max_logits, n_tok, h_q, d_qk, workspace,
                          workspace_bytes, stream);
}

smla_status sparse_mla_tree_fwd_paged(const void* q, const void* kv_pool, int64_t pool_rows,
                                      const int32_t* block_table, int max_blocks, int page_block,
                                      const int32_t* cu_seqlens_q, const int32_t* seqlens_k, int64_t n_req,
                                      const int32_t* tree_mask, int mask_words, const float* attn_sink, float sm_scale,
                                      int d_v, void* out, float* lse, float* max_logits, int64_t n_tok, int h_q, int d_qk,
                                      void* workspace, size_t workspace_bytes, smla_stream_t stream) {
  return dense_fwd<true>(q, kv_pool, pool_rows, block_table, max_blocks, page_block, cu_seqlens_q, seqlens_k, n_req, 0,
                         tree_mask, mask_words, attn_sink, sm_scale, d_v, out, lse, max_logits, n_tok, h_q, d_qk, workspace,
                         workspace_bytes, stream);
}

smla_status sparse_mla_chunk_selftest_wait_timeout(uint64_t limit_ns, smla_stream_t stream) {
  if (limit_ns == 0 || limit_ns > kWaitLimitNs) return SMLA_ERR_BAD_SHAPE;
  chunk_wait_selftest_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(limit_ns);
  return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

smla_status sparse_mla_chunk_device_status(int reset) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_chunk_status, sizeof(int)) != cudaSuccess) return SMLA_ERR_LAUNCH;
  if (reset) {
    const int z = 0;
    if (cudaMemcpyToSymbol(g_chunk_status, &z, sizeof(int)) != cudaSuccess) return SMLA_ERR_LAUNCH;
  }
  return static_cast<smla_status>(v);
}

}  // extern "C"
