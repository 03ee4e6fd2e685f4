// A speculative step around the tree attention, on the device (sm_103a): masks and positions of a tree of drafted
// tokens (sparse_mla_plan_tree), their verification against the target's probabilities (sparse_mla_verify_tree), and
// the commit of what was kept: rows moved together, pages given back (sparse_mla_commit_tree).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "../../include/sparse_mla.h"
#include "host_util.cuh"
#include "pair_ptx.cuh"

namespace smla {
namespace {

constexpr uint32_t kAll = 0xffffffffu;

// Rows of a request: cu is clamped to [0, n_tok], as in the attention over the same sums.
struct NodeRange {
  int64_t row0, n;
};
__device__ __forceinline__ NodeRange nodes_of(const int32_t* cu, int64_t b, int64_t n_tok) {
  const int64_t c0 = __ldg(cu + b), c1 = __ldg(cu + b + 1);
  NodeRange r;
  r.row0 = min(max(c0, int64_t{0}), n_tok);
  r.n = min(max(c1, r.row0), n_tok) - r.row0;
  return r;
}

// ------------------------------------------------------------------------ tree planning
// Node i of a request has the parent p_i (0 <= p_i < i, else none).  A_i = {i} + A_(p_i): what it sees of the new
// tokens; its position is the request's first new position + |A_i| - 1.
// A warp takes a request, 32 nodes at a time, a node a lane.  Within the 32, five rounds of pointer doubling give the
// set as a word (each round joins the set of the node 2^k steps up); the parent at which a chain leaves the 32 lies in
// an earlier word, whose row is complete by then.  Latency bounds it: 8 trees of 8 nodes 2.0 us, 300 of 64 2.7 us, 64 of 128
// 4.1 us, and 1.5 to 2 us for each further 32 nodes of one request (4 trees of 512: 23 us).
constexpr int kPlanWarps = 4;
constexpr int kPlanMaxCtas = 1216;
// Rows of up to so many words are written by their node's lane, longer ones a word a lane: 4 trees of 512 nodes (16 words) 23 us
// and 37; a tree of 1024 nodes 67 and 71, a chain of 1024 66 and 37.
constexpr int kLaneWords = 16;
constexpr int kMaxPlanNodes = 1 << 30;

struct TreePlanParams {
  const int32_t* parents;
  const int32_t* cu_seqlens_q;
  const int32_t* seqlens_k;
  int32_t* tree_mask;
  int32_t* positions;
  int64_t n_req, n_tok;
  int words;
};

__global__ void __launch_bounds__(32 * kPlanWarps) plan_tree_kernel(const TreePlanParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanWarps + (threadIdx.x >> 5);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanWarps;
  for (int64_t b = first; b < p.n_req; b += step) {
    const NodeRange r = nodes_of(p.cu_seqlens_q, b, p.n_tok);
    const int64_t before = max(__ldg(p.seqlens_k + b), 0) - r.n;
    int32_t ahead = lane < r.n ? __ldg(p.parents + r.row0 + lane) : -1;
    const int n = static_cast<int>(r.n);
    for (int c0 = 0; c0 < n; c0 += 32) {
      const int i = c0 + lane;
      const bool live = i < n;
      const int parent = ahead;
      ahead = i + 32 < n ? __ldg(p.parents + r.row0 + i + 32) : -1;
      const bool has = parent >= 0 && parent < i;
      uint32_t set = 1u << lane;
      int up = has && parent >= c0 ? parent - c0 : -1;    // the node 2^k steps up in these 32
      int leaves_at = has && parent < c0 ? parent : -1;
#pragma unroll
      for (int k = 0; k < 5; ++k) {
        const int from = up < 0 ? lane : up;
        const uint32_t more = __shfl_sync(kAll, set, from);
        const int out = __shfl_sync(kAll, leaves_at, from);
        const int next = __shfl_sync(kAll, up, from);
        if (up >= 0) {
          set |= more;
          leaves_at = out;
          up = next;
        }
      }
      const int word = c0 / 32;
      if (p.words <= kLaneWords) {          // a node's row by its own lane
        if (live) {
          int32_t* mask = p.tree_mask + (r.row0 + i) * p.words;
          const int32_t* above = p.tree_mask + (r.row0 + leaves_at) * p.words;
          for (int w = 0; w < p.words; ++w)
            mask[w] = w == word ? static_cast<int32_t>(set) : w < word && leaves_at >= 0 ? above[w] : 0;
        }
      } else {                              // node by node, a word a lane
        const int count = min(n - c0, 32);
        const int common = __shfl_sync(kAll, leaves_at, 0);
        const bool one_source = __all_sync(kAll, !live || leaves_at == common);   // chains, and stars
        for (int w0 = 0; w0 < p.words; w0 += 32) {
          const int w = w0 + lane;
          const bool copied = w < word && w < p.words;
          int32_t* mask = p.tree_mask + (r.row0 + c0) * p.words + w;
          const int32_t* above = p.tree_mask + r.row0 * p.words + w;
          int32_t v[32];                    // requested before any row is written
          const int32_t shared = one_source && copied && common >= 0 ? above[static_cast<int64_t>(common) * p.words] : 0;
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const int from = __shfl_sync(kAll, leaves_at, k);
            v[k] = one_source ? shared : copied && from >= 0 ? above[static_cast<int64_t>(from) * p.words] : 0;
          }
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const uint32_t own = __shfl_sync(kAll, set, k);
            if (w < p.words && k < count) mask[k * static_cast<int64_t>(p.words)] = w == word ? static_cast<int32_t>(own) : v[k];
          }
        }
      }
      if (live)
        p.positions[r.row0 + i] = static_cast<int32_t>((leaves_at >= 0 ? p.positions[r.row0 + leaves_at] + 1 : before) + __popc(set) - 1);
      __syncwarp();   // later nodes read these rows
    }
  }
  // rows of no request
  const int64_t begin = p.n_req > 0 ? min(max(static_cast<int64_t>(__ldg(p.cu_seqlens_q)), int64_t{0}), p.n_tok) : 0;
  const int64_t end = p.n_req > 0 ? min(max(static_cast<int64_t>(__ldg(p.cu_seqlens_q + p.n_req)), begin), p.n_tok) : 0;
  const int64_t spare = begin + p.n_tok - end;
  for (int64_t k = first * 32 + lane; k < spare; k += step * 32) {
    const int64_t row = k < begin ? k : end + k - begin;
    p.positions[row] = -1;
    for (int w = 0; w < p.words; ++w) p.tree_mask[row * p.words + w] = 0;
  }
}

// ------------------------------------------------------------------------ verification
// With p and q the target's and the draft's row of the current node, and x_1, x_2, .. its children's tokens (drawn from q):
//   C_1 = 0, Z_1 = 1;   r_j(v) = max(p(v) - C_j q(v), 0);   x_j is kept when u_j q(x_j) Z_j < r_j(x_j), else
//   C_(j+1) = C_j + Z_j, Z_(j+1) = sum_v r_(j+1)(v).
// This is the rule that keeps x with probability min(1, p / q) and goes on with the normalised max(p - q, 0), child by
// child; since max(max(p - a, 0) - b, 0) = max(p - a - b, 0), what is left after any number of rejections is one more
// number C, and no residual row is ever stored.  Without draft probabilities (a child is a token chosen outright, q is 1
// there): r is p without the tokens turned down, Z what they leave of 1.
// Children have larger indices than their parents, so the nodes are walked once, in order.  The last token is the first v
// with r(v_0) + .. + r(v) > u sum r.
//
// Values near that border decide which token comes out, so sums must not depend on how the row is cut: r is rounded
// to fp32 once (C too: 2^-24 of q, far below what q itself is known to), and every sum of r, Z and the comparisons with them are
// held in two floats, the second one for what the additions to the first have lost: 48 bits.  (64-bit additions run at two a
// clock and SM; the walk and the scans in 64 bits, with one more level of the search, took 3 us more.)
//
// A cluster of CTAs takes a request, each a contiguous part of the vocabulary, cut into tiles whose sums stay in shared
// memory.  All CTAs walk the tree alike; they exchange their sums only (one cluster barrier a pass).  The last token's place
// is narrowed down from the CTAs' sums to a tile's and to four values a thread, so a row is read once a pass.
//
// What bounds it.  Large batches: DRAM.  256 chains of 3 to 6 nodes over 128000 tokens, 236 MB: 45.5 us, of which 37 us are
// the rows (6.4 TB/s; 6.7 TB/s by the difference of two vocabularies) and 8 us the chain of latencies in front (sums of nodes,
// nodes, their probabilities, the walk) and behind (exchange, search).  Small ones: that chain, 5.5 us for a request of one
// node and 32000 tokens, and 2 to 3 us for each further pass (32 trees with up to five rejections at a node over 100003
// tokens: 19 to 20 us).  The first form, one CTA a request and 64-bit sums: 1 chain 25 us, 256 chains 162, 32 trees 203.  No faster:
// 16 CTAs a cluster, copies through shared memory (cp.async, 4 bytes), CTAs of 512 or 1024 threads, the warps' sums sent
// without the CTA's.
constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxVocab = 1 << 30;
constexpr int kMaxNodes = 1024;       // of a request; further ones are not tested
constexpr int kWindow = 256;          // nodes in shared memory at a time
constexpr int kMaxTiles = 256;        // of a CTA
constexpr int kTile = 4 * kVerifyThreads;   // values of a tile at most, where kMaxTiles of them are enough
constexpr int kSms = 152;             // a GB300's; the launch is fitted to them, and no result depends on it

struct VerifyParams {
  const float* target;
  const float* draft;      // or null
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* cu_seqlens_q;
  const float* accept_u;
  const float* sample_u;
  int32_t* keep;
  int32_t* out_tokens;
  int32_t* n_keep;
  int64_t target_stride, draft_stride, n_req, n_tok;
  int vocab, max_keep;
  int each, tile;            // values of a CTA, of a tile
};

// What is left of the current node's row.
struct Residual {
  const float* p;
  const float* q;           // null: r is p without the tokens in `gone`
  float c;
  const int32_t* gone;
  int n_gone;
};

__device__ __forceinline__ float left_of(const Residual& r, int v) {
  const float x = __ldg(r.p + v);
  if (r.q && r.c > 0.f) return fmaxf(fmaf(-r.c, __ldg(r.q + v), x), 0.f);
  for (int i = 0; i < r.n_gone; ++i)
    if (r.gone[i] == v) return 0.f;
  return fmaxf(x, 0.f);
}

// A sum in two floats: hi, and in lo what the additions to hi have lost (Knuth's two-sum).  64-bit additions run at 2 a clock and
// SM here.
struct __align__(8) Sum {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {
    const float s = hi + x, t = s - hi;
    lo += (hi - (s - t)) + (x - t);
    hi = s;
  }
  __device__ __forceinline__ void add(const Sum& x) {
    add(x.hi);
    lo += x.lo;
  }
  // Whether it is above x.  (The difference of the high parts is exact where they are close.)
  __device__ __forceinline__ bool above(const Sum& x) const { return (hi - x.hi) + (lo - x.lo) > 0.f; }
  __device__ __forceinline__ bool positive() const { return hi + lo > 0.f; }
};
// Over the warp: the same in every lane, and the sum up to and with a lane's own.
__device__ __forceinline__ void add_lanes(Sum& v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float hi = __shfl_xor_sync(kAll, v.hi, o), lo = __shfl_xor_sync(kAll, v.lo, o);
    const float small = fminf(v.hi, hi);
    v = {fmaxf(v.hi, hi), v.lo + lo};      // one order in both lanes
    v.add(small);
  }
}
__device__ __forceinline__ Sum upto_lane(Sum v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sum x{__shfl_up_sync(kAll, v.hi, o), __shfl_up_sync(kAll, v.lo, o)};
    if ((threadIdx.x & 31) >= o) v.add(x);
  }
  return v;
}
__device__ __forceinline__ Sum of_lane(const Sum& v, int lane) {
  return {__shfl_sync(kAll, v.hi, lane), __shfl_sync(kAll, v.lo, lane)};
}

// Four values a lane of r's row (and of q's), of the 128 from v on; 0 outside [0, end).
template <bool DRAFT, bool WIDE>
struct Step {
  float p[4], q[DRAFT ? 4 : 1];
  __device__ __forceinline__ void load(const Residual& r, int v, int end) {
    const int at = v + (WIDE ? 4 : 1) * (threadIdx.x & 31);
    if (WIDE && at >= 0 && at + 4 <= end) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(r.p + at));
      p[0] = a.x, p[1] = a.y, p[2] = a.z, p[3] = a.w;
      if (DRAFT) {
        const float4 d = __ldg(reinterpret_cast<const float4*>(r.q + at));
        q[0] = d.x, q[DRAFT ? 1 : 0] = d.y, q[DRAFT ? 2 : 0] = d.z, q[DRAFT ? 3 : 0] = d.w;
      }
      return;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int x = at + (WIDE ? 1 : 32) * u;
      const bool in = x >= 0 && x < end;
      p[u] = in ? __ldg(r.p + x) : 0.f;
      if (DRAFT) q[u] = in ? __ldg(r.q + x) : 0.f;
    }
  }
};

// Sums of r over the tiles of [v0, v1), tile values each (a multiple of 128 STEPS), into sums[0], sums[1], ..; a warp.
// STEPS steps' loads are under way, and four sums a lane are added to in turn.
template <bool DRAFT, bool WIDE, int STEPS>
__device__ __forceinline__ void tile_sums(const Residual& r, int v0, int v1, int tile, Sum* sums) {
  const int lane = threadIdx.x & 31;
  Step<DRAFT, WIDE> step[STEPS];
#pragma unroll
  for (int k = 0; k < STEPS; ++k) step[k].load(r, v0 + 128 * k, v1);
  for (int a = v0; a < v1; a += tile, ++sums) {
    const int end = min(a + tile, v1);
    Sum part[4] = {};
    for (int v = a; v < end; v += 128 * STEPS) {
      uint32_t skip = 0;               // this lane's values that are gone: bit 4 step + u
      if (!DRAFT)
        for (int i = 0; i < r.n_gone; ++i) {
          const uint32_t d = static_cast<uint32_t>(r.gone[i] - v);
          if (d < 128u * STEPS && (WIDE ? (d >> 2) & 31 : d & 31) == lane) skip |= 1u << (((d >> 7) << 2) + (WIDE ? d & 3 : (d >> 5) & 3));
        }
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {
        float x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          x[u] = fmaxf(DRAFT ? fmaf(-r.c, step[k].q[DRAFT ? u : 0], step[k].p[u]) : step[k].p[u], 0.f);
          if (!DRAFT && (skip >> (4 * k + u) & 1)) x[u] = 0.f;
        }
        step[k].load(r, v + 128 * (STEPS + k), v1);
#pragma unroll
        for (int u = 0; u < 4; ++u) part[u].add(x[u]);
      }
    }
#pragma unroll
    for (int u = 1; u < 4; ++u) part[0].add(part[u]);
    add_lanes(part[0]);
    if (lane == 0) *sums = part[0];
  }
}

// The first of n sums at which `before` + their running sum passes `target`, else the last that is above 0, else -1;
// `before` takes the sums in front of it.  One warp.
__device__ __forceinline__ int crossing(const Sum* sums, int n, const Sum& target, Sum& before) {
  const int lane = threadIdx.x & 31;
  Sum run = before;
  int last = -1;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const Sum x = i0 + lane < n ? sums[i0 + lane] : Sum{0.f, 0.f};
    Sum end = upto_lane(x), front{__shfl_up_sync(kAll, end.hi, 1), __shfl_up_sync(kAll, end.lo, 1)};
    if (lane == 0) front = {0.f, 0.f};
    end.add(run);
    front.add(run);
    const uint32_t some = __ballot_sync(kAll, x.positive()), hit = some & __ballot_sync(kAll, end.above(target));
    const int who = hit ? __ffs(hit) - 1 : some ? 31 - __clz(some) : -1;
    if (who >= 0) {
      last = i0 + who;
      before = of_lane(front, who);
    }
    if (hit) break;
    run = of_lane(end, 31);
  }
  return last;
}

enum { kWalkOn = 0, kSearch = 1, kLeave = 2 };

struct VerifyShared {
  int32_t parent[kWindow], token[kWindow], gone[kMaxNodes];
  float u[kWindow], px[kWindow], qx[kWindow];
  Sum sums[kMaxTiles];
  Sum totals[2][kMaxCluster];     // of the cluster's CTAs; of two passes in turn
  Sum target, before;
  float c;
  int cur, kept, n_gone, then, v0, v1, hit, last;
};

__device__ __forceinline__ void load_nodes(const VerifyParams& p, const NodeRange& r, int w0, int n, VerifyShared& s, int first, int step) {
  for (int i = first; i < min(n - w0, kWindow); i += step) {
    const int node = w0 + i;
    const int64_t row = r.row0 + node;
    const int32_t parent = node > 0 ? __ldg(p.parents + row) : -1, token = __ldg(p.tokens + row);
    const bool tested = parent >= 0 && parent < node && token >= 0 && token < p.vocab;   // others are never tested
    s.parent[i] = tested ? parent : -1;
    s.token[i] = token;
    s.u[i] = __ldg(p.accept_u + row);
    s.px[i] = tested ? fmaxf(__ldg(p.target + (r.row0 + parent) * p.target_stride + token), 0.f) : 0.f;
    s.qx[i] = tested && p.draft ? __ldg(p.draft + (r.row0 + parent) * p.draft_stride + token) : 1.f;
  }
}

template <int STEPS>
__global__ void __launch_bounds__(kVerifyThreads, STEPS == 4 ? 2 : STEPS == 3 ? 3 : 4) verify_tree_kernel(const VerifyParams p) {
  __shared__ VerifyShared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
  const int64_t b = blockIdx.x / ranks;
  const NodeRange r = nodes_of(p.cu_seqlens_q, b, p.n_tok);
  int32_t* keep = p.keep + b * p.max_keep;
  int32_t* out = p.out_tokens + b * p.max_keep;
  if (r.n == 0) {
    if (rank > 0) return;
    for (int i = tid; i < p.max_keep; i += kVerifyThreads) keep[i] = out[i] = -1;
    if (tid == 0) p.n_keep[b] = 0;
    return;
  }
  cluster_arrive_relaxed();    // waited for before the first sum is sent: by then every CTA runs
  const float sample_u = fmaxf(__ldg(p.sample_u + b), 0.f);
  const int n = static_cast<int>(min(r.n, static_cast<int64_t>(kMaxNodes)));
  load_nodes(p, r, 0, n, s, tid, kVerifyThreads);
  if (tid == 0) {
    s.hit = INT_MAX;
    s.last = -1;
  }
  __syncthreads();
  // the walk's state, in warp 0
  int cur = 0, kept = 1, next = 1, w0 = 0, n_gone = 0;
  float c = 0.f;
  Sum z{1.f, 0.f};
  bool summed = true;                   // Z is known
  Residual left;
  int first, behind;
  for (int pass = 0;; ++pass) {
    // ---- the walk, to its end or to where Z has to be known
    bool ask = false;
    if (warp == 0) {
      while (next < n && kept < p.max_keep) {
        if (next >= w0 + kWindow) {
          w0 += kWindow;
          __syncwarp();
          load_nodes(p, r, w0, n, s, lane, 32);
          __syncwarp();
        }
        const int i = next - w0 + lane;
        const uint32_t child = __ballot_sync(kAll, i < min(n - w0, kWindow) && s.parent[i] == cur);
        if (!child) {
          next = min(next + 32, w0 + kWindow);
          continue;
        }
        const int k = next - w0 + __ffs(child) - 1;
        if (!summed) {
          next = w0 + k;
          ask = true;
          break;
        }
        const int x = s.token[k];
        float rx = s.px[k];
        if (p.draft) {
          rx = c > 0.f ? fmaxf(fmaf(-c, s.qx[k], rx), 0.f) : rx;
        } else {
          for (int g = 0; g < n_gone; ++g)
            if (s.gone[g] == x) rx = 0.f;
        }
        // u q Z < r, the product in two floats.  Products whose rounding is recovered are rounded by name: contracted into
        // the subtraction behind it, h would not be the number whose error e holds, and the comparison one of 24 bits.
        const float uq = __fmul_rn(s.u[k], s.qx[k]), low = fmaf(s.u[k], s.qx[k], -uq);
        const float h = __fmul_rn(uq, z.hi), e = fmaf(uq, z.hi, -h) + fmaf(uq, z.lo, low * z.hi);
        if ((rx - h) - e > 0.f) {
          cur = w0 + k;
          if (lane == 0 && rank == 0) {
            keep[kept] = cur;
            out[kept - 1] = x;
          }
          ++kept;
          c = 0.f;
          z = {1.f, 0.f};
          n_gone = 0;
        } else if (p.draft) {
          z.add(c);
          c = z.hi + z.lo;
          summed = false;
        } else {
          if (lane == 0) s.gone[n_gone] = x;
          ++n_gone;
          z.add(-rx);
          if (!z.positive()) z = {0.f, 0.f};
        }
        next = w0 + k + 1;
        __syncwarp();
      }
      if (lane == 0) {
        s.cur = cur;
        s.n_gone = n_gone;
        s.c = c;
      }
    }
    __syncthreads();
    // ---- the sum of r
    left.p = p.target + (r.row0 + s.cur) * p.target_stride;
    left.c = s.c;
    left.q = left.c > 0.f ? p.draft + (r.row0 + s.cur) * p.draft_stride : nullptr;
    left.gone = s.gone;
    left.n_gone = s.n_gone;
    // 16-byte loads, where p and q lie alike: counted from the first 16-byte boundary at or in front of the row
    const bool wide = !left.q || ((reinterpret_cast<uintptr_t>(left.p) ^ reinterpret_cast<uintptr_t>(left.q)) & 15) == 0;
    first = rank * p.each - static_cast<int>(reinterpret_cast<uintptr_t>(left.p) / 4 & 3);   // this CTA's part of the vocabulary
    first = min(first, p.vocab);
    behind = min(first + p.each, p.vocab);
    const int tiles = (behind - first + p.tile - 1) / p.tile, mine = (tiles + kVerifyWarps - 1) / kVerifyWarps;
    const int v0 = min(first + warp * mine * p.tile, behind), v1 = min(v0 + mine * p.tile, behind);
    Sum* sums = s.sums + warp * mine;
    if (wide) {
      if (left.q) tile_sums<true, true, STEPS>(left, v0, v1, p.tile, sums);
      else tile_sums<false, true, STEPS>(left, v0, v1, p.tile, sums);
    } else {
      if (left.q) tile_sums<true, false, STEPS>(left, v0, v1, p.tile, sums);
      else tile_sums<false, false, STEPS>(left, v0, v1, p.tile, sums);
    }
    __syncthreads();
    if (pass == 0) cluster_wait();
    const Sum* totals = s.totals[pass & 1];
    if (warp == 0) {
      Sum sum{0.f, 0.f};
      for (int i = lane; i < tiles; i += 32) sum.add(s.sums[i]);
      add_lanes(sum);
      if (lane < ranks) store_floats(map_to_rank(smem_u32(totals + rank), lane), sum.hi, sum.lo);
      __syncwarp();
    }
    cluster_arrive();
    cluster_wait();
    if (warp == 0) {
      Sum sum = lane < ranks ? totals[lane] : Sum{0.f, 0.f};
      add_lanes(sum);
      int then = kWalkOn;
      if (ask) {
        z = sum;
        summed = true;
      } else if (sum.positive() || (c == 0.f && n_gone == 0)) {
        // the last token lies in the part of the CTA in which the running sum passes u * total
        const float h = __fmul_rn(sample_u, sum.hi);   // rounded by name, as above
        const Sum target{h, fmaf(sample_u, sum.hi, -h) + sample_u * sum.lo};
        Sum before{0.f, 0.f};
        const int owner = crossing(totals, ranks, target, before);
        then = rank == max(owner, 0) ? kSearch : kLeave;
        if (then == kSearch) {
          const int at = owner < 0 ? -1 : crossing(s.sums, tiles, target, before);
          if (lane == 0) {
            s.target = target;
            s.before = before;
            s.kept = kept;
            s.v0 = first + max(at, 0) * p.tile;
            s.v1 = at < 0 ? s.v0 : min(s.v0 + p.tile, behind);
          }
        }
      } else {   // nothing is left although p has not been used up (p <= C q everywhere): p itself
        c = 0.f;
        n_gone = 0;
        next = n;
      }
      if (lane == 0) s.then = then;
    }
    __syncthreads();
    if (s.then == kLeave) return;
    if (s.then == kSearch) break;
  }
  // ---- a tile of more than kTile values is cut again; four values of the last one a thread
  const Sum target = s.target;
  Sum before = s.before;
  int v0 = s.v0, v1 = s.v1;
  while (v1 - v0 > kTile) {
    const int part = (v1 - v0 + kVerifyWarps - 1) / kVerifyWarps, a = min(v0 + warp * part, v1), e = min(a + part, v1);
    Sum sum{0.f, 0.f};
    for (int v = max(a, 0) + lane; v < e; v += 32) sum.add(left_of(left, v));
    add_lanes(sum);
    __syncthreads();
    if (lane == 0) s.sums[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      const int at = crossing(s.sums, kVerifyWarps, target, before);
      if (lane == 0) {
        s.before = before;
        s.v0 = v0 + max(at, 0) * part;
        s.v1 = at < 0 ? s.v0 : min(s.v0 + part, v1);
      }
    }
    __syncthreads();
    before = s.before;
    v0 = s.v0;
    v1 = s.v1;
  }
  float x[4];
  Sum sum{0.f, 0.f};
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int v = v0 + 4 * tid + u;
    x[u] = v >= 0 && v < v1 ? left_of(left, v) : 0.f;
    sum.add(x[u]);
  }
  const Sum upto = upto_lane(sum);
  __syncthreads();
  if (lane == 31) s.sums[warp] = upto;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before.add(s.sums[w]);
  const Sum front{__shfl_up_sync(kAll, upto.hi, 1), __shfl_up_sync(kAll, upto.lo, 1)};
  if (lane > 0) before.add(front);
  int hit = INT_MAX, last = -1;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    before.add(x[u]);
    if (x[u] > 0.f) {
      last = v0 + 4 * tid + u;
      if (hit == INT_MAX && before.above(target)) hit = last;
    }
  }
  if (hit < INT_MAX) atomicMin(&s.hit, hit);
  if (last >= 0) atomicMax(&s.last, last);
  __syncthreads();
  const int end = s.kept;
  if (tid == 0) {
    keep[0] = 0;
    out[end - 1] = s.hit < INT_MAX ? s.hit : s.last;
    p.n_keep[b] = end;
  }
  for (int i = end + tid; i < p.max_keep; i += kVerifyThreads) keep[i] = out[i] = -1;
}

// ------------------------------------------------------------------------ commit
// Request b keeps its new tokens keep[b, 0] < keep[b, 1] < .. (n_keep[b] of them): row before + keep[i] goes to row
// before + i, in every layer.  Since keep[i] >= i, rows moved in order never overwrite one that is still to be read, and
// that holds for each 16-byte column of a row by itself: a warp takes a request of a layer, a lane the columns lane,
// lane + 32, .., four rows in flight, and no two lanes ever have to agree.
// CTA 0 does the bookkeeping instead: lengths, and the pages behind them back in front of the free list's start.
constexpr int kCommitThreads = 256;
constexpr int kRowsInFlight = 4;
// Columns of a request that a thread gives back by itself, one after the other, more of them a warp.  By threads alone, by warps alone,
// and by this rule: 86 requests of 256 that are done, up to 38 columns, 21 on average, 6.5, 16.9 and 7.9 us; 7 of 32, up to 92 columns,
// 9.6, 4.1 and 5.5; 11 of 64, up to 1631 columns, 115, 14.1 and 13.5.
constexpr int kFewColumns = 32;
constexpr int kColumnLoads = 8;       // times 32 columns that a warp looks at at once

struct CommitParams {
  const int32_t* keep;
  const int32_t* n_keep;
  const int32_t* cu_seqlens_q;
  const int32_t* seqlens_k;
  const int32_t* block_table;
  __nv_bfloat16* pool;
  int32_t* free_pages;          // null: no page is given back
  const int32_t* free_start;    // or null: n_free
  int32_t* seqlens;
  int32_t* counts;
  int64_t n_req, n_free, layer_stride, pool_rows;
  int max_keep, max_blocks, page_block, n_layers, d_qk;
};

struct Kept {
  int64_t n_k, before, n;    // length, first new position, tokens kept (-1: the request is done)
};
__device__ __forceinline__ Kept kept_of(const CommitParams& p, int64_t b) {
  const int64_t c0 = __ldg(p.cu_seqlens_q + b), c1 = __ldg(p.cu_seqlens_q + b + 1);
  const int64_t asked = __ldg(p.n_keep + b);
  Kept k;
  k.n_k = max(__ldg(p.seqlens_k + b), 0);
  const int64_t fresh = max(c1 - c0, int64_t{0});
  k.before = k.n_k - fresh;
  k.n = asked < 0 ? -1 : min(min(asked, fresh), static_cast<int64_t>(p.max_keep));
  return k;
}

__device__ __forceinline__ int64_t pool_row(const CommitParams& p, int64_t b, int64_t pos) {
  const int64_t col = pos / p.page_block;
  if (pos < 0 || col >= p.max_blocks) return -1;
  const int64_t page = __ldg(p.block_table + b * p.max_blocks + col);
  const int64_t row = page * p.page_block + (pos - col * p.page_block);
  return page < 0 || row >= p.pool_rows ? -1 : row;
}

__device__ __forceinline__ int64_t columns_of(int64_t len, const CommitParams& p) {
  return min((len + p.page_block - 1) / p.page_block, static_cast<int64_t>(p.max_blocks));
}

// Calls put(page, k) for the pages of request b's table columns [first, last), in order, k counting the mapped ones; returns how
// many there are.  By a thread, or by a warp (in every lane).
template <typename Put>
__device__ __forceinline__ int thread_pages(const CommitParams& p, int64_t b, int first, int last, Put put) {
  int count = 0;
  for (int col = first; col < last; ++col) {
    const int32_t page = __ldg(p.block_table + b * p.max_blocks + col);
    if (page >= 0) put(page, count++);
  }
  return count;
}
template <typename Put>
__device__ __forceinline__ int warp_pages(const CommitParams& p, int64_t b, int first, int last, Put put) {
  const int lane = threadIdx.x & 31;
  int count = 0;
  for (int64_t c0 = first; c0 < last; c0 += 32 * kColumnLoads) {
    int32_t page[kColumnLoads];
#pragma unroll
    for (int u = 0; u < kColumnLoads; ++u) {
      const int64_t col = c0 + 32 * u + lane;
      page[u] = col < last ? __ldg(p.block_table + b * p.max_blocks + col) : -1;
    }
#pragma unroll
    for (int u = 0; u < kColumnLoads; ++u) {
      const uint32_t mapped = __ballot_sync(kAll, page[u] >= 0);
      if (page[u] >= 0) put(page[u], count + __popc(mapped & ((1u << lane) - 1u)));
      count += __popc(mapped);
    }
  }
  return count;
}

// A thread a request.  A few columns a thread looks at by itself; requests with more (those that are done) go to the CTA's
// warps, once to be counted and once to be given back.
__device__ void commit_lengths(const CommitParams& p) {
  constexpr int kWarps = kCommitThreads / 32;
  __shared__ int64_t warp_sum[2][kWarps];
  __shared__ int64_t place[kCommitThreads];     // of a request's first page, counted down from the list's start
  __shared__ int cols[2][kCommitThreads], found[kCommitThreads], many[kCommitThreads], n_many;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t start = p.free_pages ? min(max(p.free_start ? static_cast<int64_t>(__ldg(p.free_start)) : p.n_free, int64_t{0}), p.n_free) : 0;
  int64_t pages = 0, tokens = 0;
  if (tid == 0) n_many = 0;
  for (int64_t b0 = 0; b0 < p.n_req; b0 += kCommitThreads) {
    __syncthreads();
    const int64_t b = b0 + tid;
    Kept k{0, 0, 0};
    int first = 0, last = 0;
    if (b < p.n_req) {
      k = kept_of(p, b);
      const int64_t len = k.n < 0 ? 0 : max(k.before + k.n, int64_t{0});
      p.seqlens[b] = static_cast<int32_t>(len);
      first = static_cast<int>(columns_of(len, p));
      last = p.free_pages ? static_cast<int>(columns_of(k.n_k, p)) : first;
    }
    const bool few = last - first <= kFewColumns;
    if (few) {
      found[tid] = thread_pages(p, b, first, last, [](int32_t, int) {});
    } else {
      cols[0][tid] = first;
      cols[1][tid] = last;
      many[atomicAdd(&n_many, 1)] = tid;        // in any order: each has its own place
    }
    __syncthreads();
    for (int i = warp; i < n_many; i += kWarps) {
      const int of = many[i], n = warp_pages(p, b0 + of, cols[0][of], cols[1][of], [](int32_t, int) {});
      if (lane == 0) found[of] = n;
    }
    __syncthreads();
    const int64_t back = found[tid];
    int64_t end = back, kept = max(k.n, int64_t{0});
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(kAll, end, o), t = __shfl_up_sync(kAll, kept, o);
      if (lane >= o) {
        end += u;
        kept += t;
      }
    }
    if (lane == 31) {
      warp_sum[0][warp] = end;
      warp_sum[1][warp] = kept;
    }
    __syncthreads();
    int64_t at = pages + end - back;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += warp_sum[0][w];
      pages += warp_sum[0][w];
      tokens += warp_sum[1][w];
    }
    const auto give_back = [&](int64_t place_of, int32_t page, int n) {
      const int64_t to = start - 1 - (place_of + n);
      if (to >= 0) p.free_pages[to] = page;
    };
    place[tid] = at;
    if (few) thread_pages(p, b, first, last, [&](int32_t page, int n) { give_back(at, page, n); });
    __syncthreads();
    for (int i = warp; i < n_many; i += kWarps) {
      const int of = many[i];
      warp_pages(p, b0 + of, cols[0][of], cols[1][of], [&](int32_t page, int n) { give_back(place[of], page, n); });
    }
    __syncthreads();
    if (tid == 0) n_many = 0;
  }
  if (tid == 0) {
    const int64_t given = min(pages, start);
    p.counts[0] = static_cast<int32_t>(min(tokens, static_cast<int64_t>(INT32_MAX)));
    p.counts[1] = static_cast<int32_t>(start - given);
    p.counts[2] = static_cast<int32_t>(min(pages - given, static_cast<int64_t>(INT32_MAX)));
  }
}

__global__ void __launch_bounds__(kCommitThreads) commit_tree_kernel(const CommitParams p) {
  if (blockIdx.x == 0) {
    commit_lengths(p);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) - 1) * (kCommitThreads / 32) + (threadIdx.x >> 5);
  if (unit >= p.n_req * p.n_layers) return;
  const int64_t b = unit / p.n_layers, layer = unit % p.n_layers;
  // the first entries of keep are requested beside the lengths that say how many of them count
  int64_t from = lane < p.max_keep ? __ldg(p.keep + b * p.max_keep + lane) : -1;
  const Kept k = kept_of(p, b);
  __nv_bfloat16* pool = p.pool + layer * p.layer_stride;
  const int pieces = p.d_qk / 8;
  for (int64_t i0 = 0; i0 < k.n; i0 += 32) {
    const int64_t i = i0 + lane;
    int64_t src = -1, dst = -1;
    if (i < k.n) {
      if (i0 > 0) from = __ldg(p.keep + b * p.max_keep + i);
      if (from > i && from < k.n_k - k.before) {
        src = pool_row(p, b, k.before + from);
        dst = pool_row(p, b, k.before + i);
      }
    }
    uint32_t todo = __ballot_sync(kAll, src >= 0 && dst >= 0);
    while (todo) {
      int64_t row[kRowsInFlight], to[kRowsInFlight];
#pragma unroll
      for (int x = 0; x < kRowsInFlight; ++x) {
        const int who = todo ? __ffs(todo) - 1 : 0;
        row[x] = __shfl_sync(kAll, src, who);
        to[x] = todo ? __shfl_sync(kAll, dst, who) : -1;
        todo &= todo - 1;
      }
      uint4 v[3][kRowsInFlight];
#pragma unroll
      for (int u = 0; u < 3; ++u)
#pragma unroll
        for (int x = 0; x < kRowsInFlight; ++x)
          if (to[x] >= 0 && lane + 32 * u < pieces) v[u][x] = reinterpret_cast<const uint4*>(pool + row[x] * p.d_qk)[lane + 32 * u];
#pragma unroll
      for (int u = 0; u < 3; ++u)
#pragma unroll
        for (int x = 0; x < kRowsInFlight; ++x)
          if (to[x] >= 0 && lane + 32 * u < pieces) reinterpret_cast<uint4*>(pool + to[x] * p.d_qk)[lane + 32 * u] = v[u][x];
    }
  }
}

}  // namespace
}  // namespace smla

using namespace smla;

extern "C" {

smla_status sparse_mla_plan_tree(const int32_t* parents, const int32_t* cu_seqlens_q, const int32_t* seqlens_k,
                                 int32_t* tree_mask, int32_t* positions, int64_t n_req, int64_t n_tok, int mask_words,
                                 smla_stream_t stream) {
  if (n_req < 0 || n_req > INT32_MAX || n_tok < 0 || n_tok > kMaxPlanNodes || mask_words < 1 || mask_words > 1024)
    return SMLA_ERR_BAD_SHAPE;
  if (n_tok == 0) return SMLA_OK;
  if (!parents || !tree_mask || !positions || (n_req > 0 && (!cu_seqlens_q || !seqlens_k))) return SMLA_ERR_NULL_PTR;
  for (const void* x : {static_cast<const void*>(parents), static_cast<const void*>(cu_seqlens_q),
                        static_cast<const void*>(seqlens_k), static_cast<const void*>(tree_mask), static_cast<const void*>(positions)})
    if (!aligned_to(x, 4)) return SMLA_ERR_MISALIGNED;
  const size_t reqs = static_cast<size_t>(n_req) * 4, toks = static_cast<size_t>(n_tok) * 4;
  const Span in[] = {{parents, toks}, {cu_seqlens_q, reqs + 4}, {seqlens_k, reqs}};
  const Span written[] = {{tree_mask, toks * mask_words}, {positions, toks}};
  if (any_overlap(in, written)) return SMLA_ERR_BAD_SHAPE;
  const TreePlanParams p{parents, cu_seqlens_q, seqlens_k, tree_mask, positions, n_req, n_tok, mask_words};
  int64_t ctas = (n_req + kPlanWarps - 1) / kPlanWarps;
  ctas = ctas < 1 ? 1 : ctas > kPlanMaxCtas ? kPlanMaxCtas : ctas;
  plan_tree_kernel<<<static_cast<unsigned>(ctas), 32 * kPlanWarps, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

smla_status sparse_mla_verify_tree(const float* target_probs, int64_t target_stride, const float* draft_probs,
                                   int64_t draft_stride, const int32_t* tokens, const int32_t* parents,
                                   const int32_t* cu_seqlens_q, const float* accept_u, const float* sample_u,
                                   int32_t* keep, int32_t* out_tokens, int32_t* n_keep, int64_t n_req, int64_t n_tok,
                                   int vocab, int max_keep, smla_stream_t stream) {
  if (n_req < 0 || n_req > INT32_MAX || n_tok < 0 || n_tok > INT32_MAX || vocab < 1 || vocab > kMaxVocab ||
      max_keep < 1 || n_req > INT32_MAX / max_keep)
    return SMLA_ERR_BAD_SHAPE;
  if (n_req == 0) return SMLA_OK;
  if (!cu_seqlens_q || !sample_u || !keep || !out_tokens || !n_keep ||
      (n_tok > 0 && (!target_probs || !tokens || !parents || !accept_u)))
    return SMLA_ERR_NULL_PTR;
  if (n_tok < 2) target_stride = draft_stride = vocab;   // the stride of a single row is not looked at
  if (target_stride < vocab || (draft_probs && draft_stride < vocab) || target_stride > INT64_MAX / 8 / (n_tok + 1) ||
      (draft_probs && draft_stride > INT64_MAX / 8 / (n_tok + 1)))
    return SMLA_ERR_BAD_SHAPE;
  const void* all[] = {target_probs, draft_probs, tokens, parents, cu_seqlens_q, accept_u, sample_u, keep, out_tokens, n_keep};
  for (const void* x : all)
    if (!aligned_to(x, 4)) return SMLA_ERR_MISALIGNED;
  const size_t reqs = static_cast<size_t>(n_req) * 4, toks = static_cast<size_t>(n_tok) * 4;
  const size_t t_bytes = n_tok > 0 ? (static_cast<size_t>(n_tok - 1) * target_stride + vocab) * 4 : 0;
  const size_t d_bytes = n_tok > 0 && draft_probs ? (static_cast<size_t>(n_tok - 1) * draft_stride + vocab) * 4 : 0;
  const Span in[] = {{target_probs, t_bytes}, {draft_probs, d_bytes}, {tokens, toks}, {parents, toks},
                     {cu_seqlens_q, reqs + 4}, {accept_u, toks}, {sample_u, reqs}};
  const Span written[] = {{keep, reqs * max_keep}, {out_tokens, reqs * max_keep}, {n_keep, reqs}};
  if (any_overlap(in, written)) return SMLA_ERR_BAD_SHAPE;
  VerifyParams p{target_probs, draft_probs, tokens, parents, cu_seqlens_q, accept_u, sample_u, keep, out_tokens,
                 n_keep, target_stride, draft_stride, n_req, n_tok, vocab, max_keep, 0, 0};
  // CTAs a request, and steps of loads under way: four where two CTAs an SM are enough, three for three, two for four.  Clusters of
  // four and more do not fill the GPU to the last place (they fall 16 or 64 short, found by trial), and what does not fit runs after
  // the rest.  Chains of 3 to 6 nodes with the draft's rows over 128000 tokens, in us, (CTAs, steps), the chosen pair first:
  // 48 requests 13.8 (8, 3), 14.5 (8, 2), 14.8 (4, 4); 76 requests 20.0 (4, 3), 21.3 (4, 2), 22.2 (2, 4), 27.1 (4, 4), which just does
  // not fit; 128 requests 27.0 (2, 4), 26.8 (4, 2); 152 requests 30.5 (2, 4), 31.6 (2, 3), 34.6 (2, 2), 41.3 (4, 2); 200 requests
  // 38.3 (2, 3), 39.8 (2, 2), 40.6 (1, 4); 256 requests 45.5 (1, 4), 45.9 (2, 2), 48.1 (1, 3), 56.2 (1, 2); 400 requests 65.1 (1, 3),
  // 68.0 (1, 2), 80.1 (1, 4); 512 requests 80.4 (1, 2), 87.0 (1, 4), 100.3 (1, 3).  One request of one node over 32000 tokens
  // 5.5 (8, 4), 5.9 (4, 4), 6.9 (2, 4), 8.4 (1, 4).
  const auto fits = [&](int r, int steps) {
    return r * n_req <= kSms * (steps == 4 ? 2 : steps == 3 ? 3 : 4) - (r < 4 ? 0 : r == 4 || steps == 4 ? 16 : 64);
  };
  const auto room = [&](int r) { return r < kMaxCluster && vocab > r * kTile; };
  int ranks = 1, steps = fits(1, 4) ? 4 : fits(1, 3) ? 3 : 2;
  if (steps == 4) {
    while (room(ranks) && fits(2 * ranks, 4)) ranks *= 2;
    if (room(ranks) && ranks * n_req <= 3 * kSms / 2) {
      ranks *= 2;
      steps = fits(ranks, 3) ? 3 : 2;
    }
  }
  p.each = ((vocab + 3 + ranks - 1) / ranks + 3) / 4 * 4;
  p.tile = (p.each + kVerifyWarps - 1) / kVerifyWarps;
  const int most = kTile / (128 * steps) * (128 * steps);
  p.tile = p.tile > most ? most : p.tile;
  if (p.each > p.tile * kMaxTiles) p.tile = (p.each + kMaxTiles - 1) / kMaxTiles;
  p.tile = (p.tile + 128 * steps - 1) / (128 * steps) * (128 * steps);
  cudaLaunchAttribute cluster{};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = ranks;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  if (n_req > INT32_MAX / ranks) return SMLA_ERR_BAD_SHAPE;
  cfg.gridDim = dim3(static_cast<unsigned>(n_req * ranks));
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cfg.attrs = &cluster;
  cfg.numAttrs = 1;
  const auto kernel = steps == 4 ? verify_tree_kernel<4> : steps == 3 ? verify_tree_kernel<3> : verify_tree_kernel<2>;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

smla_status sparse_mla_commit_tree(const int32_t* keep, const int32_t* n_keep, int max_keep, const int32_t* cu_seqlens_q,
                                   const int32_t* seqlens_k, const int32_t* block_table, int max_blocks, int page_block,
                                   int64_t n_req, void* kv_pool, int n_layers, int64_t layer_stride, int64_t pool_rows,
                                   int d_qk, int32_t* free_pages, int64_t n_free, const int32_t* free_start,
                                   int32_t* seqlens, int32_t* counts, smla_stream_t stream) {
  if (n_req < 0 || n_req > INT32_MAX || max_keep < 1 || n_req > INT32_MAX / max_keep || max_blocks < 1 || page_block < 1 ||
      static_cast<int64_t>(max_blocks) * page_block > INT32_MAX || n_layers < 0 || pool_rows < 0 || pool_rows > INT32_MAX ||
      n_free < 0 || n_free > INT32_MAX || (n_layers > 0 && d_qk != 512 && d_qk != 576))
    return SMLA_ERR_BAD_SHAPE;
  if (pool_rows == 0) n_layers = 0;
  if (n_layers == 1) layer_stride = 0;                   // the stride of a single layer is not looked at
  if (n_layers > 1 && (layer_stride < pool_rows * d_qk || layer_stride > INT64_MAX / 4 / n_layers)) return SMLA_ERR_BAD_SHAPE;
  if (!counts || (n_req > 0 && (!keep || !n_keep || !cu_seqlens_q || !seqlens_k || !block_table || !seqlens)) ||
      (n_layers > 0 && !kv_pool))
    return SMLA_ERR_NULL_PTR;
  const void* all[] = {keep, n_keep, cu_seqlens_q, seqlens_k, block_table, free_pages, free_start, seqlens, counts};
  for (const void* x : all)
    if (!aligned_to(x, 4)) return SMLA_ERR_MISALIGNED;
  if (n_layers > 0 && (!aligned_to(kv_pool, 16) || layer_stride % 8)) return SMLA_ERR_MISALIGNED;
  const size_t reqs = static_cast<size_t>(n_req) * 4;
  const size_t pool_bytes = n_layers > 0 ? (static_cast<size_t>(n_layers - 1) * layer_stride + static_cast<size_t>(pool_rows) * d_qk) * 2 : 0;
  const Span in[] = {{keep, reqs * max_keep}, {n_keep, reqs}, {cu_seqlens_q, reqs + 4}, {seqlens_k, reqs},
                     {block_table, reqs * max_blocks}, {free_start, 4}};
  const Span written[] = {{kv_pool, pool_bytes}, {free_pages, static_cast<size_t>(n_free) * 4}, {seqlens, reqs}, {counts, 12}};
  if (any_overlap(in, written)) return SMLA_ERR_BAD_SHAPE;
  const int64_t per_cta = kCommitThreads / 32, ctas = 1 + (n_req * n_layers + per_cta - 1) / per_cta;
  if (ctas > INT32_MAX) return SMLA_ERR_BAD_SHAPE;
  const CommitParams p{keep, n_keep, cu_seqlens_q, seqlens_k, block_table, static_cast<__nv_bfloat16*>(kv_pool),
                       n_free > 0 ? free_pages : nullptr,
                       free_start, seqlens, counts, n_req, n_free, layer_stride, pool_rows, max_keep, max_blocks,
                       page_block, n_layers, d_qk};
  commit_tree_kernel<<<static_cast<unsigned>(ctas), kCommitThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

}  // extern "C"
