// A speculative step around the tree attention, on the device (sm_103a): masks and positions of a tree of drafted
// tokens (sparse_mla_plan_tree), their verification against the target's probabilities (sparse_mla_verify_tree), and
// the commit of what was kept: rows moved together, pages given back (sparse_mla_commit_tree).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "../../include/sparse_mla.h"
#include "host_util.cuh"

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
// an earlier word, whose row is complete by then.
constexpr int kPlanWarps = 4;
constexpr int kPlanMaxCtas = 1216;

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
    for (int64_t c0 = 0; c0 < r.n; c0 += 32) {
      const int64_t i = c0 + lane;
      const bool live = i < r.n;
      const int64_t parent = live ? __ldg(p.parents + r.row0 + i) : -1;
      const bool has = parent >= 0 && parent < i;
      uint32_t set = 1u << lane;
      int up = has && parent >= c0 ? static_cast<int>(parent - c0) : -1;    // the node 2^k steps up in these 32
      int64_t leaves_at = has && parent < c0 ? parent : -1;
#pragma unroll
      for (int k = 0; k < 5; ++k) {
        const int from = up < 0 ? lane : up;
        const uint32_t more = __shfl_sync(kAll, set, from);
        const int64_t out = __shfl_sync(kAll, leaves_at, from);
        const int next = __shfl_sync(kAll, up, from);
        if (up >= 0) {
          set |= more;
          leaves_at = out;
          up = next;
        }
      }
      if (live) {
        const int64_t row = r.row0 + i;
        int32_t* mask = p.tree_mask + row * p.words;
        const int32_t* above = p.tree_mask + (r.row0 + leaves_at) * p.words;
        for (int64_t w = 0; w < p.words; ++w)
          mask[w] = w == c0 / 32 ? static_cast<int32_t>(set) : w < c0 / 32 && leaves_at >= 0 ? above[w] : 0;
        p.positions[row] = static_cast<int32_t>((leaves_at >= 0 ? p.positions[r.row0 + leaves_at] + 1 : before) + __popc(set) - 1);
      }
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
// to fp32 once (C too: 2^-24 of q, far below what q itself is known to), and sums of r are held in two floats per lane
// (the rounding error of each addition is added up beside the sum) and in 64 bits from there on.
constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxNodes = 1024;       // of a request; further ones are not tested
constexpr int kScanLen = 256;         // a range that one warp searches

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
};

// What is left of the current node's row.
struct Residual {
  const float* p;
  const float* q;           // null: r is p without the tokens in `gone`
  float c;
  const int32_t* gone;
  int n_gone;
};

__device__ __forceinline__ float left_of(const Residual& r, int64_t v) {
  const float x = __ldg(r.p + v);
  if (r.q && r.c > 0.f) return fmaxf(fmaf(-r.c, __ldg(r.q + v), x), 0.f);
  for (int i = 0; i < r.n_gone; ++i)
    if (r.gone[i] == v) return 0.f;
  return fmaxf(x, 0.f);
}

// Sum of r over [v0, v1), in every lane.
__device__ __forceinline__ double sum_of(const Residual& r, int64_t v0, int64_t v1) {
  float hi = 0.f, lo = 0.f;
  for (int64_t v = v0 + (threadIdx.x & 31); v < v1; v += 32) {
    const float x = left_of(r, v);
    const float s = hi + x, t = s - hi;
    lo += (hi - (s - t)) + (x - t);     // what the addition lost
    hi = s;
  }
  double sum = static_cast<double>(hi) + lo;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  return sum;
}

struct VerifyShared {
  int32_t parent[kMaxNodes], token[kMaxNodes], gone[kMaxNodes];
  float u[kMaxNodes], px[kMaxNodes], qx[kMaxNodes];
  double sums[kVerifyWarps];
  double z;
  float c;
  int cur, kept, next, n_gone, ask;
  int64_t v0, v1;
  double before;
};

// The first of n sums at which base + their running sum passes `target`, else the last that is above 0, else -1;
// `before` becomes base + the sums in front of it.  One warp.
__device__ __forceinline__ int crossing(const double* sums, int n, double target, double& before) {
  const int lane = threadIdx.x & 31;
  double run = before;
  int last = -1;
  double at_last = run;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const double x = i0 + lane < n ? sums[i0 + lane] : 0.0;
    double end = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double u = __shfl_up_sync(kAll, end, o);
      if (lane >= o) end += u;
    }
    const uint32_t hit = __ballot_sync(kAll, i0 + lane < n && x > 0.0 && run + end > target);
    const uint32_t some = __ballot_sync(kAll, x > 0.0);
    const int who = hit ? __ffs(hit) - 1 : some ? 31 - __clz(some) : -1;
    if (who >= 0) {
      last = i0 + who;
      at_last = run + __shfl_sync(kAll, end - x, who);
    }
    if (hit) break;
    run += __shfl_sync(kAll, end, 31);
  }
  before = at_last;
  return last;
}

__global__ void __launch_bounds__(kVerifyThreads) verify_tree_kernel(const VerifyParams p) {
  __shared__ VerifyShared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t b = blockIdx.x;
  const NodeRange r = nodes_of(p.cu_seqlens_q, b, p.n_tok);
  int32_t* keep = p.keep + b * p.max_keep;
  int32_t* out = p.out_tokens + b * p.max_keep;
  if (r.n == 0) {
    for (int i = tid; i < p.max_keep; i += kVerifyThreads) keep[i] = out[i] = -1;
    if (tid == 0) p.n_keep[b] = 0;
    return;
  }
  const int n = static_cast<int>(min(r.n, static_cast<int64_t>(kMaxNodes)));
  for (int i = tid; i < n; i += kVerifyThreads) {
    const int64_t row = r.row0 + i;
    const int32_t parent = i > 0 ? __ldg(p.parents + row) : -1, token = __ldg(p.tokens + row);
    const bool tested = parent >= 0 && parent < i && token >= 0 && token < p.vocab;   // others are never tested
    s.parent[i] = tested ? parent : -1;
    s.token[i] = token;
    s.u[i] = __ldg(p.accept_u + row);
    s.px[i] = tested ? fmaxf(__ldg(p.target + (r.row0 + parent) * p.target_stride + token), 0.f) : 0.f;
    s.qx[i] = tested && p.draft ? __ldg(p.draft + (r.row0 + parent) * p.draft_stride + token) : 1.f;
  }
  if (tid == 0) {
    s.cur = 0;
    s.kept = s.next = 1;
    s.c = 0.f;
    s.z = 1.0;
    s.n_gone = 0;
  }
  __syncthreads();
  Residual left;
  for (;;) {
    // ---- the walk, to its end or to where Z has to be known
    if (warp == 0) {
      int cur = s.cur, kept = s.kept, next = s.next, n_gone = s.n_gone;
      float c = s.c;
      double z = s.z;                   // below 0: not summed yet
      bool ask = false;
      while (next < n && kept < p.max_keep) {
        const int i = next + lane;
        const uint32_t child = __ballot_sync(kAll, i < n && s.parent[i] == cur);
        if (!child) {
          next += 32;
          continue;
        }
        const int k = next + __ffs(child) - 1;
        if (z < 0.0) {
          next = k;
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
        if (static_cast<double>(s.u[k]) * s.qx[k] * z < rx) {
          if (lane == 0) {
            keep[kept] = k;
            out[kept - 1] = x;
          }
          cur = k;
          ++kept;
          c = 0.f;
          z = 1.0;
          n_gone = 0;
        } else if (p.draft) {
          c = static_cast<float>(c + z);
          z = -1.0;
        } else {
          if (lane == 0) s.gone[n_gone] = x;
          ++n_gone;
          z -= rx;
          if (z < 0.0) z = 0.0;
        }
        next = k + 1;
        __syncwarp();
      }
      __syncwarp();
      if (lane == 0) {
        s.cur = cur;
        s.kept = kept;
        s.next = next;
        s.n_gone = n_gone;
        s.c = c;
        s.z = z;
        s.ask = ask;
      }
    }
    __syncthreads();
    // ---- the sum of r
    left.p = p.target + (r.row0 + s.cur) * p.target_stride;
    left.q = p.draft ? p.draft + (r.row0 + s.cur) * p.draft_stride : nullptr;
    left.c = s.c;
    left.gone = s.gone;
    left.n_gone = s.n_gone;
    const int64_t each = (static_cast<int64_t>(p.vocab) + kVerifyWarps - 1) / kVerifyWarps;
    const double mine = sum_of(left, min(warp * each, static_cast<int64_t>(p.vocab)), min((warp + 1) * each, static_cast<int64_t>(p.vocab)));
    if (lane == 0) s.sums[warp] = mine;
    __syncthreads();
    double total = 0.0;
    for (int w = 0; w < kVerifyWarps; ++w) total += s.sums[w];
    if (s.ask) {
      __syncthreads();
      if (tid == 0) s.z = total;
      __syncthreads();
      continue;
    }
    if (total > 0.0 || (left.c == 0.f && left.n_gone == 0)) {
      // ---- the last token: the range in which the running sum passes u * total, cut again until a warp searches it
      const double target = static_cast<double>(fmaxf(__ldg(p.sample_u + b), 0.f)) * total;
      int64_t v0 = 0, v1 = p.vocab, part = each;
      double before = 0.0;
      for (;;) {
        if (warp == 0) {
          const int at = crossing(s.sums, kVerifyWarps, target, before);
          if (lane == 0) {
            s.v0 = at < 0 ? -1 : v0 + at * part;
            s.v1 = at < 0 ? -1 : min(v0 + (at + 1) * part, v1);
            s.before = before;
          }
        }
        __syncthreads();
        v0 = s.v0;
        v1 = s.v1;
        before = s.before;
        if (v1 - v0 <= kScanLen) break;
        part = (v1 - v0 + kVerifyWarps - 1) / kVerifyWarps;
        const double sub = sum_of(left, min(v0 + warp * part, v1), min(v0 + (warp + 1) * part, v1));
        __syncthreads();
        if (lane == 0) s.sums[warp] = sub;
        __syncthreads();
      }
      if (warp == 0) {
        int64_t token = -1;
        for (int64_t a = v0; a >= 0 && a < v1; a += 32) {
          const float x = a + lane < v1 ? left_of(left, a + lane) : 0.f;
          double end = x;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const double u = __shfl_up_sync(kAll, end, o);
            if (lane >= o) end += u;
          }
          const uint32_t hit = __ballot_sync(kAll, x > 0.f && before + end > target);
          const uint32_t some = __ballot_sync(kAll, x > 0.f);
          if (hit) {
            token = a + __ffs(hit) - 1;
            break;
          }
          if (some) token = a + 31 - __clz(some);
          before += __shfl_sync(kAll, end, 31);
        }
        const int kept = s.kept;
        if (lane == 0) {
          keep[0] = 0;
          out[kept - 1] = static_cast<int32_t>(token);
          p.n_keep[b] = kept;
        }
        for (int i = kept + lane; i < p.max_keep; i += 32) keep[i] = out[i] = -1;
      }
      return;
    }
    // nothing is left although p has not been used up (p <= C q everywhere): p itself
    __syncthreads();
    if (tid == 0) {
      s.c = 0.f;
      s.n_gone = 0;
      s.next = n;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------ commit
// Request b keeps its new tokens keep[b, 0] < keep[b, 1] < .. (n_keep[b] of them): row before + keep[i] goes to row
// before + i, in every layer.  Since keep[i] >= i, rows moved in order never overwrite one that is still to be read, and
// that holds for each 16-byte column of a row by itself: a warp takes a request of a layer, a lane the columns lane,
// lane + 32, .., four rows in flight, and no two lanes ever have to agree.
// CTA 0 does the bookkeeping instead: lengths, and the pages behind them back in front of the free list's start.
constexpr int kCommitThreads = 256;
constexpr int kRowsInFlight = 4;

struct CommitParams {
  const int32_t* keep;
  const int32_t* n_keep;
  const int32_t* cu_seqlens_q;
  const int32_t* seqlens_k;
  const int32_t* block_table;
  __nv_bfloat16* pool;
  int32_t* free_pages;          // or null: no page is given back
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

__device__ void commit_lengths(const CommitParams& p) {
  __shared__ int64_t warp_sum[2][kCommitThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t start = p.free_pages ? min(max(p.free_start ? static_cast<int64_t>(__ldg(p.free_start)) : p.n_free, int64_t{0}), p.n_free) : 0;
  int64_t pages = 0, tokens = 0;
  for (int64_t b0 = 0; b0 < p.n_req; b0 += kCommitThreads) {
    const int64_t b = b0 + tid;
    Kept k{0, 0, 0};
    int64_t first = 0, last = 0, back = 0;
    if (b < p.n_req) {
      k = kept_of(p, b);
      const int64_t len = k.n < 0 ? 0 : max(k.before + k.n, int64_t{0});
      p.seqlens[b] = static_cast<int32_t>(len);
      first = columns_of(len, p);
      last = p.free_pages ? columns_of(k.n_k, p) : first;
      for (int64_t col = first; col < last; ++col) back += __ldg(p.block_table + b * p.max_blocks + col) >= 0;
    }
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
    for (int w = 0; w < kCommitThreads / 32; ++w) {
      if (w < warp) at += warp_sum[0][w];
      pages += warp_sum[0][w];
      tokens += warp_sum[1][w];
    }
    for (int64_t col = first; col < last; ++col) {
      const int32_t page = __ldg(p.block_table + b * p.max_blocks + col);
      if (page < 0) continue;
      if (at < start) p.free_pages[start - 1 - at] = page;
      ++at;
    }
    __syncthreads();
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
  const Kept k = kept_of(p, b);
  __nv_bfloat16* pool = p.pool + layer * p.layer_stride;
  const int pieces = p.d_qk / 8;
  for (int64_t i0 = 0; i0 < k.n; i0 += 32) {
    const int64_t i = i0 + lane;
    int64_t src = -1, dst = -1;
    if (i < k.n) {
      const int64_t from = __ldg(p.keep + b * p.max_keep + i);
      if (from > i && from < k.n_k - k.before) {
        src = pool_row(p, b, k.before + from);
        dst = pool_row(p, b, k.before + i);
      }
    }
    uint32_t todo = __ballot_sync(kAll, src >= 0 && dst >= 0);
    while (todo) {
      int64_t from[kRowsInFlight], to[kRowsInFlight];
#pragma unroll
      for (int x = 0; x < kRowsInFlight; ++x) {
        const int who = todo ? __ffs(todo) - 1 : 0;
        from[x] = __shfl_sync(kAll, src, who);
        to[x] = todo ? __shfl_sync(kAll, dst, who) : -1;
        todo &= todo - 1;
      }
      for (int c = lane; c < pieces; c += 32) {
        uint4 v[kRowsInFlight];
#pragma unroll
        for (int x = 0; x < kRowsInFlight; ++x)
          if (to[x] >= 0) v[x] = reinterpret_cast<const uint4*>(pool + from[x] * p.d_qk)[c];
#pragma unroll
        for (int x = 0; x < kRowsInFlight; ++x)
          if (to[x] >= 0) reinterpret_cast<uint4*>(pool + to[x] * p.d_qk)[c] = v[x];
      }
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
  if (n_req < 0 || n_req > INT32_MAX || n_tok < 0 || n_tok > INT32_MAX || mask_words < 1 || mask_words > 1024)
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
  if (n_req < 0 || n_req > INT32_MAX || n_tok < 0 || n_tok > INT32_MAX || vocab < 1 || max_keep < 1 ||
      n_req > INT32_MAX / max_keep)
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
  const VerifyParams p{target_probs, draft_probs, tokens, parents, cu_seqlens_q, accept_u, sample_u, keep, out_tokens,
                       n_keep, target_stride, draft_stride, n_req, n_tok, vocab, max_keep};
  verify_tree_kernel<<<static_cast<unsigned>(n_req), kVerifyThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
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
  const CommitParams p{keep, n_keep, cu_seqlens_q, seqlens_k, block_table, static_cast<__nv_bfloat16*>(kv_pool), free_pages,
                       free_start, seqlens, counts, n_req, n_free, layer_stride, pool_rows, max_keep, max_blocks,
                       page_block, n_layers, d_qk};
  commit_tree_kernel<<<static_cast<unsigned>(ctas), kCommitThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

}  // extern "C"
