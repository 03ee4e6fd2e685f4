// Bookkeeping of a paged latent cache on the device (sm_103a): which pages and rows a step's new
// tokens get (sparse_mla_plan_pages), and the write of their rows (sparse_mla_append_kv).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/sparse_mla.h"
#include "host_util.cuh"

namespace smla {
namespace {

// ------------------------------------------------------------------------ page planning
// For request b with o_b cached and m_b new tokens (both taken as 0 when negative):
//   e_b   = min(sum_{i<=b} m_i, n_tokens), cu = [0, e_0, e_1, ...]; c_b = cu[b+1] - cu[b]
//   len_b = o_b + c_b
//   new pages: table columns ceil(o_b / P) .. ceil(len_b / P) - 1 (below max_blocks), filled from the
//   free list in order of (request, column)
//   token t of request b: position o_b + t - cu[b], slot table[b][pos / P] * P + pos % P
// One launch.  Every CTA scans all requests in chunks of kPlanThreads (two block scans: tokens and
// pages), so no CTA waits for another; the tokens, pages and requests themselves are dealt to the
// CTAs in blocks of kPlanThreads, and a token (page) finds its request by a binary search in the
// chunk's running sums.  Nothing that one CTA writes is read by another: a token in a page that
// this launch hands out computes the page from the free list instead of reading the table.
// The work is a few loads deep: latency bounds it, not bytes, so a CTA takes about one token a thread (700 requests with
// 37 k tokens: 8 us, with eight tokens a thread 14 us; 1024 threads and requests a chunk are no faster.  256
// requests of one token: 4.3 us, 8 requests: 3.0 us).
constexpr int kPlanThreads = 256;
constexpr int kPlanMaxCtas = 152;

struct PlanParams {
  const int32_t* seqlens;
  const int32_t* new_lens;
  int32_t* block_table;
  const int32_t* free_pages;
  const int32_t* free_start;   // or null: 0
  int32_t* seqlens_k;
  int32_t* cu_seqlens_q;
  int32_t* slots;
  int32_t* positions;
  int32_t* counts;
  int64_t n_req;
  int64_t n_free;
  int32_t n_tokens;
  int32_t max_blocks;
  int32_t page_block;
};

struct PlanChunk {
  int64_t page_end[kPlanThreads];   // running sum of new pages over all requests so far, inclusive
  int32_t tok_end[kPlanThreads];    // the same of tokens, clamped to n_tokens
  int32_t tok_begin[kPlanThreads];
  int32_t old_len[kPlanThreads];
  int32_t first[kPlanThreads];      // first new table column
  int64_t warp_sum[2][kPlanThreads / 32];
};

// Inclusive scan over the CTA.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w)
    if (w < warp) v += warp_sum[w];
  return v;
}

// First i with end[i] > x.  The caller knows that there is one among the n entries.
template <typename T>
__device__ __forceinline__ int owner_of(const T* end, int n, T x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// ceil(len / page_block), at most max_blocks; max_blocks * page_block fits 31 bits.
__device__ __forceinline__ int32_t blocks_of(int64_t len, int32_t page_block, int32_t max_blocks) {
  if (len >= static_cast<int64_t>(max_blocks) * page_block) return max_blocks;
  return static_cast<int32_t>((static_cast<uint32_t>(len) + page_block - 1u) / static_cast<uint32_t>(page_block));
}

__global__ void __launch_bounds__(kPlanThreads) plan_pages_kernel(const PlanParams p) {
  __shared__ PlanChunk c;
  const int tid = threadIdx.x;
  const int64_t grid = gridDim.x, cta = blockIdx.x;
  const int64_t start0 = p.free_start ? max(__ldg(p.free_start), 0) : 0;
  auto free_page = [&](int64_t k) -> int32_t {   // k-th page that this call hands out
    const int64_t i = start0 + k;
    return i < p.n_free ? __ldg(p.free_pages + i) : -1;
  };
  int64_t tok_run = 0, page_run = 0;
  if (cta == 0 && tid == 0) p.cu_seqlens_q[0] = 0;
  for (int64_t r0 = 0; r0 < p.n_req; r0 += kPlanThreads) {
    const int n = static_cast<int>(min(static_cast<int64_t>(kPlanThreads), p.n_req - r0));
    const int64_t r = r0 + tid;
    const int32_t old_len = tid < n ? max(__ldg(p.seqlens + r), 0) : 0;
    const int32_t fresh = tid < n ? max(__ldg(p.new_lens + r), 0) : 0;
    const int64_t incl = tok_run + block_scan(fresh, c.warp_sum[0]);
    const int32_t end = static_cast<int32_t>(min(incl, static_cast<int64_t>(p.n_tokens)));
    const int32_t begin = static_cast<int32_t>(min(incl - fresh, static_cast<int64_t>(p.n_tokens)));
    const int64_t len = static_cast<int64_t>(old_len) + (end - begin);
    const int32_t first = blocks_of(old_len, p.page_block, p.max_blocks);
    const int32_t need = tid < n ? blocks_of(len, p.page_block, p.max_blocks) - first : 0;
    const int64_t page_end = page_run + block_scan(need, c.warp_sum[1]);
    c.page_end[tid] = page_end;
    c.tok_end[tid] = end;
    c.tok_begin[tid] = begin;
    c.old_len[tid] = old_len;
    c.first[tid] = first;
    if (tid < n && (r0 / kPlanThreads) % grid == cta) {
      p.seqlens_k[r] = static_cast<int32_t>(min(len, static_cast<int64_t>(INT32_MAX)));
      p.cu_seqlens_q[r + 1] = end;
    }
    __syncthreads();
    const int64_t tok_next = c.tok_end[kPlanThreads - 1], page_next = c.page_end[kPlanThreads - 1];
    // the chunk's tokens: block t / kPlanThreads belongs to CTA (t / kPlanThreads) % grid
    if (tok_run < tok_next) {
      const int64_t b0 = tok_run / kPlanThreads;
      for (int64_t b = b0 + (cta - b0 % grid + grid) % grid; b * kPlanThreads < tok_next; b += grid) {
        const int64_t t = b * kPlanThreads + tid;
        if (t < tok_run || t >= tok_next) continue;
        const int i = owner_of(c.tok_end, n, static_cast<int32_t>(t));
        const int64_t pos = static_cast<int64_t>(c.old_len[i]) + (t - c.tok_begin[i]);
        int64_t slot = -1;
        const int32_t col = pos <= INT32_MAX ? static_cast<int32_t>(pos) / p.page_block : p.max_blocks;
        if (col < p.max_blocks) {
          const int32_t page = col < c.first[i]
                                   ? p.block_table[(r0 + i) * p.max_blocks + col]
                                   : free_page((i > 0 ? c.page_end[i - 1] : page_run) + (col - c.first[i]));
          slot = page < 0 ? -1 : static_cast<int64_t>(page) * p.page_block + (pos - static_cast<int64_t>(col) * p.page_block);
          if (slot > INT32_MAX) slot = -1;
        }
        p.slots[t] = static_cast<int32_t>(slot);
        p.positions[t] = static_cast<int32_t>(min(pos, static_cast<int64_t>(INT32_MAX)));
      }
    }
    // the chunk's new pages, dealt in the same way
    if (page_run < page_next) {
      const int64_t b0 = page_run / kPlanThreads;
      for (int64_t b = b0 + (cta - b0 % grid + grid) % grid; b * kPlanThreads < page_next; b += grid) {
        const int64_t k = b * kPlanThreads + tid;
        if (k < page_run || k >= page_next) continue;
        const int i = owner_of(c.page_end, n, k);
        const int64_t col = c.first[i] + (k - (i > 0 ? c.page_end[i - 1] : page_run));
        p.block_table[(r0 + i) * p.max_blocks + col] = free_page(k);
      }
    }
    tok_run = tok_next;
    page_run = page_next;
    __syncthreads();   // the chunk's arrays are rewritten
  }
  for (int64_t t = tok_run + cta * kPlanThreads + tid; t < p.n_tokens; t += grid * kPlanThreads) {
    p.slots[t] = -1;
    p.positions[t] = -1;
  }
  if (cta == 0 && tid == 0) {
    const int64_t room = max(p.n_free - start0, static_cast<int64_t>(0));
    const int64_t taken = min(page_run, room);
    p.counts[0] = static_cast<int32_t>(tok_run);
    p.counts[1] = static_cast<int32_t>(start0 + taken);
    p.counts[2] = static_cast<int32_t>(min(page_run - taken, static_cast<int64_t>(INT32_MAX)));
  }
}

// ------------------------------------------------------------------------ row append
// Row of token t in the pool: [ y | turned rope columns ] with
//   y_d = c_d * rsqrt(mean(c^2) + eps) * w_d   (or c_d without a norm weight),
//   (x_2i, x_2i+1) -> (x_2i cos_i - x_2i+1 sin_i, x_2i+1 cos_i + x_2i sin_i),
// cos_i, sin_i from the row of the rope table at the token's position.  The same launch turns the
// queries' rope columns of every head into q[..., 512:].  All arithmetic is in fp32 and each value
// is rounded to bf16 once.  Every input is read once and every output written once.  Latency bounds it: a
// warp does one unit behind two dependent reads (position, then table row), and 58-60 % of the warp slots are
// active.  8192 tokens, 16 heads, 54 MB: 12.3 us over inputs that pass the L2 (4.4 TB/s; DRAM at 27-30 % of its
// peak in the launch, since the rows written stay in the L2), 9.8 us over two sets that it holds; 256 tokens, 128
// heads, 9 MB: 4.2 and 2.7 us.
// A warp takes one unit: the token's row (16 latent values a lane, the sum of squares over the
// warp), or 16 heads of its queries (8 lanes a head, 16 bytes a lane, four loads in flight).
constexpr int kAppendThreads = 256;
constexpr int kLatent = 512;
constexpr int kRope = 64;
constexpr int kHeadsPerUnit = 16;

struct AppendParams {
  const __nv_bfloat16* c_kv;
  const __nv_bfloat16* k_pe;        // or null
  const int32_t* slots;
  const int32_t* positions;         // with rope
  const float* rope;                // [max_pos, 64]: cos | sin; or null
  const __nv_bfloat16* norm_weight; // or null
  const __nv_bfloat16* q_pe;        // or null
  __nv_bfloat16* q;
  __nv_bfloat16* pool;
  int32_t* past_rope;               // or null
  int64_t c_stride, k_stride, q_stride_t, q_stride_h;   // elements
  int64_t max_pos, pool_rows, n;
  float eps;
  int d_qk, h_q, units;             // units of a token: 1 + head groups
};

__device__ __forceinline__ float2 unpack(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t turn(uint32_t v, float cs, float sn) {
  const float2 x = unpack(v);
  return pack(x.x * cs - x.y * sn, x.y * cs + x.x * sn);
}

__device__ __forceinline__ void append_row(const AppendParams& p, int64_t t, int64_t pos, int lane) {
  const int64_t slot = __ldg(p.slots + t);
  if (slot < 0 || slot >= p.pool_rows) return;
  const uint4* src = reinterpret_cast<const uint4*>(p.c_kv + t * p.c_stride);
  uint4 v[2] = {__ldg(src + lane), __ldg(src + 32 + lane)};
  uint32_t pe = 0;
  float cs = 1.f, sn = 0.f;
  if (p.k_pe) {
    pe = __ldg(reinterpret_cast<const uint32_t*>(p.k_pe + t * p.k_stride) + lane);
    if (p.rope) {
      cs = __ldg(p.rope + pos * kRope + lane);
      sn = __ldg(p.rope + pos * kRope + kRope / 2 + lane);
    }
  }
  uint4* dst = reinterpret_cast<uint4*>(p.pool + slot * p.d_qk);
  if (p.norm_weight) {
    const uint4* wsrc = reinterpret_cast<const uint4*>(p.norm_weight);
    const uint4 w[2] = {__ldg(wsrc + lane), __ldg(wsrc + 32 + lane)};
    uint32_t* vv = reinterpret_cast<uint32_t*>(v);
    const uint32_t* ww = reinterpret_cast<const uint32_t*>(w);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = unpack(vv[i]);
      sum = fmaf(x.x, x.x, fmaf(x.y, x.y, sum));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = rsqrtf(sum * (1.f / kLatent) + p.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = unpack(vv[i]), y = unpack(ww[i]);
      vv[i] = pack(x.x * inv * y.x, x.y * inv * y.y);
    }
  }
  dst[lane] = v[0];
  dst[32 + lane] = v[1];
  if (p.k_pe) reinterpret_cast<uint32_t*>(p.pool + slot * p.d_qk + kLatent)[lane] = p.rope ? turn(pe, cs, sn) : pe;
}

__device__ __forceinline__ void turn_heads(const AppendParams& p, int64_t t, int64_t pos, int h0, int lane) {
  const int part = lane & 7;   // 8 of the 64 columns: pairs 4 part .. 4 part + 3
  const float4 cs = __ldg(reinterpret_cast<const float4*>(p.rope + pos * kRope) + part);
  const float4 sn = __ldg(reinterpret_cast<const float4*>(p.rope + pos * kRope + kRope / 2) + part);
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int h = h0 + 4 * i + (lane >> 3);
    if (h < p.h_q) v[i] = reinterpret_cast<const uint4*>(p.q_pe + t * p.q_stride_t + h * p.q_stride_h)[part];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int h = h0 + 4 * i + (lane >> 3);
    if (h < p.h_q) {
      const uint4 o = make_uint4(turn(v[i].x, cs.x, sn.x), turn(v[i].y, cs.y, sn.y), turn(v[i].z, cs.z, sn.z),
                                 turn(v[i].w, cs.w, sn.w));
      reinterpret_cast<uint4*>(p.q + (t * p.h_q + h) * p.d_qk + kLatent)[part] = o;
    }
  }
}

__global__ void __launch_bounds__(kAppendThreads) append_kv_kernel(const AppendParams p) {
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (unit >= p.n * p.units) return;
  const int64_t t = unit / p.units;
  const int u = static_cast<int>(unit % p.units);
  int64_t pos = 0;
  if (p.rope) {
    pos = __ldg(p.positions + t);
    if (pos < 0 || pos >= p.max_pos) {   // padding, or behind the table: nothing is written for it
      // a count, so the order of the additions does not matter
      if (pos >= 0 && u == 0 && lane == 0 && p.past_rope) atomicAdd(p.past_rope, 1);
      return;
    }
  }
  if (u == 0) append_row(p, t, pos, lane);
  else turn_heads(p, t, pos, (u - 1) * kHeadsPerUnit, lane);
}

smla_status append_kv(const void* c_kv, int64_t c_stride, const void* k_pe, int64_t k_stride, const int32_t* slots,
                      const int32_t* positions, const float* rope, int64_t max_pos, const void* norm_weight, float eps,
                      const void* q_pe, int64_t q_stride_t, int64_t q_stride_h, void* q, int h_q, void* kv_pool,
                      int64_t pool_rows, int d_qk, int64_t n, int32_t* past_rope, smla_stream_t stream) {
  if (n < 0 || n > INT32_MAX || pool_rows < 0 || pool_rows > INT32_MAX || (d_qk != kLatent && d_qk != kLatent + kRope) ||
      !std::isfinite(eps) || eps < 0.f)
    return SMLA_ERR_BAD_SHAPE;
  const bool roped = d_qk > kLatent;
  // rope columns exist exactly when d_qk is 576; a rotation needs them, its positions and its table
  if ((k_pe != nullptr) != roped && n > 0) return SMLA_ERR_NULL_PTR;
  if (rope && (!roped || max_pos < 1)) return SMLA_ERR_BAD_SHAPE;
  if (rope && !positions && n > 0) return SMLA_ERR_NULL_PTR;
  if ((q_pe != nullptr) != (q != nullptr) || (q_pe && !rope)) return SMLA_ERR_NULL_PTR;
  if (q_pe && (h_q < 1 || h_q > 1024)) return SMLA_ERR_BAD_SHAPE;
  if (n == 0) return SMLA_OK;
  if (!c_kv || !slots || (pool_rows > 0 && !kv_pool)) return SMLA_ERR_NULL_PTR;
  // the stride of a single token or head addresses nothing, whatever it is
  if (n == 1) c_stride = k_stride = q_stride_t = 0;
  if (h_q == 1) q_stride_h = 0;
  if (c_stride < 0 || k_stride < 0 || q_stride_t < 0 || q_stride_h < 0) return SMLA_ERR_BAD_SHAPE;
  if (!aligned_to(c_kv, 16) || c_stride % 8 || !aligned_to(k_pe, 4) || k_stride % 2 || !aligned_to(norm_weight, 16) ||
      !aligned_to(rope, 16) || !aligned_to(q_pe, 16) || q_stride_t % 8 || q_stride_h % 8 || !aligned_to(q, 16) ||
      !aligned_to(kv_pool, 16) || !aligned_to(slots, 4) || !aligned_to(positions, 4) || !aligned_to(past_rope, 4))
    return SMLA_ERR_MISALIGNED;
  // rows are written while others are still read; the queries' columns may be turned where they are
  const size_t pool_bytes = static_cast<size_t>(pool_rows) * d_qk * 2;
  const size_t q_bytes = static_cast<size_t>(n) * (q ? h_q : 0) * d_qk * 2;
  const size_t c_bytes = (static_cast<size_t>(n - 1) * c_stride + kLatent) * 2;
  const size_t k_bytes = (static_cast<size_t>(n - 1) * k_stride + kRope) * 2;
  const size_t q_pe_bytes =
      q ? (static_cast<size_t>(n - 1) * q_stride_t + static_cast<size_t>(h_q - 1) * q_stride_h + kRope) * 2 : 0;
  const bool in_place = q_pe == static_cast<const __nv_bfloat16*>(q) + kLatent && (n == 1 || q_stride_t == int64_t{h_q} * d_qk) &&
                        (h_q == 1 || q_stride_h == d_qk);
  const size_t ints = static_cast<size_t>(n) * 4;
  const Span in[] = {{c_kv, c_bytes}, {k_pe, k_bytes}, {slots, ints}, {rope ? positions : nullptr, ints},
                     {rope, static_cast<size_t>(max_pos) * kRope * 4}, {norm_weight, kLatent * 2},
                     {in_place ? nullptr : q_pe, q_pe_bytes}};
  const Span written[] = {{kv_pool, pool_bytes}, {q, q_bytes}, {past_rope, 4}};
  if (any_overlap(in, written)) return SMLA_ERR_BAD_SHAPE;
  AppendParams p{};
  p.c_kv = static_cast<const __nv_bfloat16*>(c_kv);
  p.k_pe = static_cast<const __nv_bfloat16*>(k_pe);
  p.slots = slots;
  p.positions = positions;
  p.rope = rope;
  p.norm_weight = static_cast<const __nv_bfloat16*>(norm_weight);
  p.q_pe = static_cast<const __nv_bfloat16*>(q_pe);
  p.q = static_cast<__nv_bfloat16*>(q);
  p.pool = static_cast<__nv_bfloat16*>(kv_pool);
  p.past_rope = past_rope;
  p.c_stride = c_stride;
  p.k_stride = k_stride;
  p.q_stride_t = q_stride_t;
  p.q_stride_h = q_stride_h;
  p.max_pos = max_pos;
  p.pool_rows = pool_rows;
  p.n = n;
  p.eps = eps;
  p.d_qk = d_qk;
  p.h_q = h_q;
  p.units = 1 + (q_pe ? (h_q + kHeadsPerUnit - 1) / kHeadsPerUnit : 0);
  const int64_t per_cta = kAppendThreads / 32;
  const int64_t ctas = (n * p.units + per_cta - 1) / per_cta;
  if (ctas > INT32_MAX) return SMLA_ERR_BAD_SHAPE;
  append_kv_kernel<<<static_cast<unsigned>(ctas), kAppendThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

}  // namespace
}  // namespace smla

using namespace smla;

extern "C" {

smla_status sparse_mla_plan_pages(const int32_t* seqlens, const int32_t* new_lens, int32_t* block_table,
                                  const int32_t* free_pages, const int32_t* free_start, int32_t* seqlens_k,
                                  int32_t* cu_seqlens_q, int32_t* slots, int32_t* positions, int32_t* counts,
                                  int64_t n_req, int64_t n_free, int64_t n_tokens, int max_blocks, int page_block,
                                  smla_stream_t stream) {
  if (n_req < 0 || n_req > INT32_MAX || n_free < 0 || n_free > INT32_MAX || n_tokens < 0 || n_tokens > INT32_MAX ||
      max_blocks < 1 || page_block < 1 || static_cast<int64_t>(max_blocks) * page_block > INT32_MAX)
    return SMLA_ERR_BAD_SHAPE;
  if (!cu_seqlens_q || !counts || (n_req > 0 && (!seqlens || !new_lens || !block_table || !seqlens_k)) ||
      (n_free > 0 && !free_pages) || (n_tokens > 0 && (!slots || !positions)))
    return SMLA_ERR_NULL_PTR;
  const void* all[] = {seqlens, new_lens, block_table, free_pages, free_start, seqlens_k, cu_seqlens_q, slots,
                       positions, counts};
  for (const void* x : all)
    if (!aligned_to(x, 4)) return SMLA_ERR_MISALIGNED;
  // the CTAs read the inputs while others write the outputs: those must be other memory
  const size_t rb = static_cast<size_t>(n_req) * 4, tb = static_cast<size_t>(n_tokens) * 4;
  const Span in[] = {{seqlens, rb}, {new_lens, rb}, {free_start, 4}, {free_pages, static_cast<size_t>(n_free) * 4}};
  const Span written[] = {{block_table, rb * max_blocks}, {seqlens_k, rb}, {cu_seqlens_q, rb + 4},
                          {slots, tb}, {positions, tb}, {counts, 12}};
  if (any_overlap(in, written)) return SMLA_ERR_BAD_SHAPE;
  PlanParams p{seqlens, new_lens, block_table, free_pages, free_start, seqlens_k, cu_seqlens_q, slots, positions,
               counts, n_req, n_free, static_cast<int32_t>(n_tokens), max_blocks, page_block};
  int64_t ctas = (n_tokens + kPlanThreads - 1) / kPlanThreads;
  ctas = ctas < 1 ? 1 : ctas > kPlanMaxCtas ? kPlanMaxCtas : ctas;
  plan_pages_kernel<<<static_cast<unsigned>(ctas), kPlanThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

smla_status sparse_mla_append_kv(const void* c_kv, int64_t c_stride, const void* k_pe, int64_t k_stride,
                                 const int32_t* slots, const int32_t* positions, const float* rope, int64_t max_pos,
                                 const void* norm_weight, float eps, const void* q_pe, int64_t q_stride_t,
                                 int64_t q_stride_h, void* q, int h_q, void* kv_pool, int64_t pool_rows, int d_qk,
                                 int64_t n, smla_stream_t stream) {
  return append_kv(c_kv, c_stride, k_pe, k_stride, slots, positions, rope, max_pos, norm_weight, eps, q_pe, q_stride_t,
                   q_stride_h, q, h_q, kv_pool, pool_rows, d_qk, n, nullptr, stream);
}

smla_status sparse_mla_append_kv_counted(const void* c_kv, int64_t c_stride, const void* k_pe, int64_t k_stride,
                                         const int32_t* slots, const int32_t* positions, const float* rope,
                                         int64_t max_pos, const void* norm_weight, float eps, const void* q_pe,
                                         int64_t q_stride_t, int64_t q_stride_h, void* q, int h_q, void* kv_pool,
                                         int64_t pool_rows, int d_qk, int64_t n, int32_t* past_rope,
                                         smla_stream_t stream) {
  if (!past_rope) return SMLA_ERR_NULL_PTR;
  return append_kv(c_kv, c_stride, k_pe, k_stride, slots, positions, rope, max_pos, norm_weight, eps, q_pe, q_stride_t,
                   q_stride_h, q, h_q, kv_pool, pool_rows, d_qk, n, past_rope, stream);
}

}  // extern "C"
