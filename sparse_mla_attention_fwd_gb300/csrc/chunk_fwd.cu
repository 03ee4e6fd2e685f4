// Dense MLA attention of a chunk of new tokens over a paged latent cache (sm_103a).
//
// Request b has q_b new tokens (rows cu[b] .. cu[b+1]-1 of q) and L_b keys in the cache, its new
// tokens' own rows among them.  Token i of the request stands at position L_b - q_b + i and sees
// the keys at positions j <= that (causal) or every j < L_b.  With K = row[:d_qk], V = row[:512]:
//   s_j = sm_scale <q, K_j>, m = max s_j, l = sum exp(s_j - m),
//   O = sum exp(s_j - m) V_j / (l + [sink] exp(sink_h - m)), lse = m + ln l, max_logits = m.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/sparse_mla.h"
#include "host_util.cuh"

namespace smla {
namespace {

constexpr int kDv = 512;
constexpr float kLog2e = 1.4426950408889634f;

struct ChunkParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* pool;
  const int32_t* block_table;
  const int32_t* cu_seqlens_q;
  const int32_t* seqlens_k;
  const float* attn_sink;   // or null
  __nv_bfloat16* out;
  float* lse;
  float* max_logits;
  int64_t pool_rows, n_req, n_tok;
  float sm_scale;
  int h_q, max_blocks, page_block, causal;
};

// One CTA per (token, eight heads), one warp per head; 32 keys a step, one key per lane for the
// scores, 16 value columns per lane for the output.
constexpr int kHeads = 8;
constexpr int kKeys = 32;

template <int D_QK>
__global__ void __launch_bounds__(32 * kHeads) chunk_fwd_kernel(const ChunkParams p) {
  constexpr int kPitch = D_QK + 8;
  extern __shared__ uint8_t smem[];
  __nv_bfloat16* sk = reinterpret_cast<__nv_bfloat16*>(smem);
  float* sq = reinterpret_cast<float*>(smem + kKeys * kPitch * 2);
  __shared__ int64_t s_row[kKeys];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y * kHeads + warp;
  // the request of this token: the last one that starts at or before it
  int64_t lo = 0, hi = p.n_req;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (p.cu_seqlens_q[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int64_t begin = p.cu_seqlens_q[lo], end = p.cu_seqlens_q[lo + 1];
  if (t < begin || t >= end) return;   // no request's token: its rows are left as they are
  const int64_t n_k = max(p.seqlens_k[lo], 0);
  int64_t seen = p.causal ? n_k - (end - begin) + (t - begin) + 1 : n_k;
  seen = min(max(seen, static_cast<int64_t>(0)), static_cast<int64_t>(p.max_blocks) * p.page_block);
  const bool live = h < p.h_q;
  for (int d = lane; d < D_QK; d += 32)
    sq[warp * D_QK + d] = live ? __bfloat162float(p.q[(t * p.h_q + h) * D_QK + d]) : 0.f;
  float m = -INFINITY, l = 0.f, o[16] = {};
  for (int64_t k0 = 0; k0 < seen; k0 += kKeys) {
    __syncthreads();
    if (tid < kKeys) {
      const int64_t j = k0 + tid;
      int64_t row = -1;
      if (j < seen) {
        const int64_t page = p.block_table[lo * p.max_blocks + j / p.page_block];
        row = page < 0 ? -1 : page * p.page_block + j % p.page_block;
        if (row >= p.pool_rows) row = -1;
      }
      s_row[tid] = row;
    }
    __syncthreads();
    for (int e = tid; e < kKeys * (D_QK / 8); e += 32 * kHeads) {
      const int j = e / (D_QK / 8), d = e % (D_QK / 8);
      const uint4 v = s_row[j] < 0 ? make_uint4(0, 0, 0, 0)
                                   : reinterpret_cast<const uint4*>(p.pool + s_row[j] * D_QK)[d];
      *reinterpret_cast<uint4*>(sk + j * kPitch + 8 * d) = v;
    }
    __syncthreads();
    float s = 0.f;
    for (int d = 0; d < D_QK; ++d) s = fmaf(sq[warp * D_QK + d], __bfloat162float(sk[lane * kPitch + d]), s);
    s = s_row[lane] < 0 ? -INFINITY : s * p.sm_scale;
    float top = s;
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    top = fmaxf(top, m);
    const float base = top == -INFINITY ? 0.f : top;
    const float keep = exp2f((m - base) * kLog2e);
    const float e = exp2f((s - base) * kLog2e);
    float sum = e;
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = l * keep + sum;
    m = top;
    for (int i = 0; i < 16; ++i) o[i] *= keep;
    for (int j = 0; j < kKeys; ++j) {
      const float w = __shfl_sync(0xffffffffu, e, j);
      for (int i = 0; i < 8; ++i) {
        const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(sk + j * kPitch + 64 * i + 2 * lane));
        o[2 * i] = fmaf(w, v.x, o[2 * i]);
        o[2 * i + 1] = fmaf(w, v.y, o[2 * i + 1]);
      }
    }
  }
  if (!live) return;
  const bool empty = !(l > 0.f);
  const float den = p.attn_sink ? l + exp2f((p.attn_sink[h] - m) * kLog2e) : l;
  const float inv = empty ? 0.f : 1.f / den;
  const int64_t r = t * p.h_q + h;
  for (int i = 0; i < 8; ++i) {
    const float a = empty ? 0.f : o[2 * i] * inv, b = empty ? 0.f : o[2 * i + 1] * inv;
    *reinterpret_cast<__nv_bfloat162*>(p.out + r * kDv + 64 * i + 2 * lane) = __floats2bfloat162_rn(a, b);
  }
  if (lane == 0) {
    p.lse[r] = empty ? INFINITY : m + logf(l);
    p.max_logits[r] = empty ? -INFINITY : m;
  }
}

template <int D_QK>
smla_status launch(const ChunkParams& p, cudaStream_t stream) {
  const int smem = kKeys * (D_QK + 8) * 2 + kHeads * D_QK * 4;
  if (cudaFuncSetAttribute(chunk_fwd_kernel<D_QK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return SMLA_ERR_LAUNCH;
  chunk_fwd_kernel<D_QK><<<dim3(static_cast<unsigned>(p.n_tok), (p.h_q + kHeads - 1) / kHeads), 32 * kHeads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

}  // namespace
}  // namespace smla

using namespace smla;

extern "C" {

size_t sparse_mla_chunk_workspace_size(int64_t n_tok, int h_q) {
  (void)n_tok;
  (void)h_q;
  return 0;
}

smla_status sparse_mla_chunk_fwd_paged(const void* q, const void* kv_pool, int64_t pool_rows,
                                       const int32_t* block_table, int max_blocks, int page_block,
                                       const int32_t* cu_seqlens_q, const int32_t* seqlens_k, int64_t n_req, int causal,
                                       const float* attn_sink, float sm_scale, int d_v, void* out, float* lse,
                                       float* max_logits, int64_t n_tok, int h_q, int d_qk, void* workspace,
                                       size_t workspace_bytes, smla_stream_t stream) {
  if (n_tok < 0 || n_req < 0 || n_req > INT32_MAX || h_q < 1 || h_q > 1024 || (d_qk != 512 && d_qk != 576) ||
      d_v != kDv || !(sm_scale > 0.f) || !std::isfinite(sm_scale) || n_tok > INT32_MAX / h_q)
    return SMLA_ERR_BAD_SHAPE;
  if (n_tok == 0 || n_req == 0) return SMLA_OK;
  if (pool_rows < 1 || pool_rows > INT32_MAX || max_blocks < 1 || page_block < 1 ||
      static_cast<int64_t>(max_blocks) * page_block > INT32_MAX)
    return SMLA_ERR_BAD_SHAPE;
  if (!q || !kv_pool || !block_table || !cu_seqlens_q || !seqlens_k || !out || !lse || !max_logits)
    return SMLA_ERR_NULL_PTR;
  if (!aligned_to(q, 16) || !aligned_to(kv_pool, 16) || !aligned_to(out, 16) || !aligned_to(lse, 4) ||
      !aligned_to(max_logits, 4) || !aligned_to(block_table, 4) || !aligned_to(cu_seqlens_q, 4) ||
      !aligned_to(seqlens_k, 4) || !aligned_to(attn_sink, 4))
    return SMLA_ERR_MISALIGNED;
  if (workspace_bytes < sparse_mla_chunk_workspace_size(n_tok, h_q)) return SMLA_ERR_WORKSPACE;
  (void)workspace;
  ChunkParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.pool = static_cast<const __nv_bfloat16*>(kv_pool);
  p.block_table = block_table;
  p.cu_seqlens_q = cu_seqlens_q;
  p.seqlens_k = seqlens_k;
  p.attn_sink = attn_sink;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.max_logits = max_logits;
  p.pool_rows = pool_rows;
  p.n_req = n_req;
  p.n_tok = n_tok;
  p.sm_scale = sm_scale;
  p.h_q = h_q;
  p.max_blocks = max_blocks;
  p.page_block = page_block;
  p.causal = causal != 0;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return d_qk == 512 ? launch<512>(p, s) : launch<576>(p, s);
}

}  // extern "C"
