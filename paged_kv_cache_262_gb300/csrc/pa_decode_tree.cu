// Decode attention of trees of drafted tokens over the paged cache, for
// sm_103a: every node of every sequence's tree attends the sequence's context
// and its own chain of ancestors,
//   out = sum_j softmax_j(scale * q.k_j) v_j,  j < c and j = c + a, a on the chain.
// It serves the decode phase of "Configuring vLLM and PagedAttention for High
// Throughput Enterprise LLM Serving" ("Memory Bottlenecks in Autoregressive
// LLM Inference": decode reads the whole cache for every token): the tokens of
// a tree share one reading of it.
//
// A CTA per (node, kv head): its four warps take the keys in turn, a lane
// D / 32 of a key's dimensions, each of the kv head's query heads with its own
// running maximum and sum in fp32; the warps' states are joined at the end.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "pa_internal.h"
#include "pa_ptx.cuh"
#include "pa_tree.cuh"
#include "pagedattn.h"

namespace pa {
namespace {

struct TreeArgs {
  const __nv_bfloat16 *q, *k, *v;
  const int32_t *bt, *ctx, *cu, *parents;
  __nv_bfloat16 *out;
  int32_t *err;
  int S, Hq, Hkv, G, B, num_blocks, max_blocks, max_ctx, max_nodes, total;
  float scale_log2;
};

constexpr int kTrWarps = 4;

template <int D>
__global__ void __launch_bounds__(kTrWarps * 32) tree_kernel(const TreeArgs a) {
  constexpr int E = D / 32;
  __shared__ int chain[PA_MAX_TREE_NODES];
  __shared__ int len;
  __shared__ float so[kTrWarps][16][D], sm[kTrWarps][16], sl[kTrWarps][16];
  const int i = blockIdx.x, h = blockIdx.y, s = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const TreeRange r = tree_range(a.cu, s, a.total, a.max_nodes);
  if (r.bad && tid == 0 && a.err) atomicOr(a.err, PA_DEVERR_TREE);
  if (i >= r.count) return;
  const int c = __ldg(a.ctx + s);
  const bool room = c >= 0 && c <= a.max_ctx - r.count && c <= a.max_blocks * a.B - r.count;
  if (tid == 0) {
    int n = 0, at = i;
    if (r.bad || !room) {
      at = -1;
      if (!room && !r.bad && a.err) atomicOr(a.err, PA_DEVERR_CTX);
    }
    while (at >= 0) {
      chain[n++] = at;
      const int p = __ldg(a.parents + r.first + at);
      if (!good_parent(at, p)) {
        if (a.err) atomicOr(a.err, PA_DEVERR_TREE);
        n = 0;
        break;
      }
      at = p;
    }
    len = n;
  }
  __syncthreads();
  // (a tree past max_nodes has rows past the grid: they are zeros too)
  if (len == 0) {
    for (int row = i; row < r.count; row += a.max_nodes)
      for (int d = tid; d < a.G * D; d += kTrWarps * 32)
        a.out[((size_t)(r.first + row) * a.Hq + (size_t)h * a.G) * D + d] = __float2bfloat16(0.f);
    return;
  }
  const int keys = c + len;
  float q[16][E], o[16][E], m[16], l[16];
#pragma unroll
  for (int g = 0; g < 16; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[g][e] = 0.f;
      q[g][e] = g < a.G ? __bfloat162float(
                              a.q[((size_t)(r.first + i) * a.Hq + (size_t)h * a.G + g) * D + lane * E + e])
                        : 0.f;
    }
  }
  for (int j = warp; j < keys; j += kTrWarps) {
    const int pos = j < c ? j : c + chain[j - c];
    const int pg = __ldg(a.bt + (size_t)s * a.max_blocks + pos / a.B);
    if (pg < 0 || pg >= a.num_blocks) {
      if (lane == 0 && a.err) atomicOr(a.err, PA_DEVERR_PAGE);
      continue;
    }
    const size_t at = (((size_t)pg * a.Hkv + h) * a.B + pos % a.B) * D + lane * E;
    float k[E], v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      k[e] = __bfloat162float(a.k[at + e]);
      v[e] = __bfloat162float(a.v[at + e]);
    }
#pragma unroll
    for (int g = 0; g < 16; ++g) {
      if (g >= a.G) break;
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) x += q[g][e] * k[e];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      x *= a.scale_log2;
      const float mn = fmaxf(m[g], x), base = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m[g] - base), p = exp2f(x - base);
      m[g] = mn;
      l[g] = l[g] * f + p;
#pragma unroll
      for (int e = 0; e < E; ++e) o[g][e] = o[g][e] * f + (p == 0.f ? 0.f : p * v[e]);
    }
  }
#pragma unroll
  for (int g = 0; g < 16; ++g) {
    if (g >= a.G) break;
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][g][lane * E + e] = o[g][e];
    if (lane == 0) sm[warp][g] = m[g], sl[warp][g] = l[g];
  }
  __syncthreads();
  for (int idx = tid; idx < a.G * D; idx += kTrWarps * 32) {
    const int g = idx / D, d = idx % D;
    float mx = -INFINITY, den = 0.f, acc = 0.f;
    for (int w = 0; w < kTrWarps; ++w) mx = fmaxf(mx, sm[w][g]);
    const float base = mx == -INFINITY ? 0.f : mx;
    for (int w = 0; w < kTrWarps; ++w) {
      const float f = exp2f(sm[w][g] - base);
      den += sl[w][g] * f;
      acc += so[w][g][d] * f;
    }
    a.out[((size_t)(r.first + i) * a.Hq + (size_t)h * a.G) * D + idx] =
        __float2bfloat16(den != 0.f ? acc / den : 0.f);
  }
}

int validate_tree(const pa_decode_desc *d, int max_nodes) {
  const int st = validate_decode_desc(d);
  if (st != PA_OK) return st;
  if (max_nodes <= 0) return PA_ERR_INVALID;
  return max_nodes > PA_MAX_TREE_NODES ? PA_ERR_UNSUPPORTED : PA_OK;
}

}  // namespace
}  // namespace pa

extern "C" size_t pa_decode_tree_workspace_bytes(const pa_decode_desc *d, int max_tree_nodes) {
  using namespace pa;
  if (validate_tree(d, max_tree_nodes) != PA_OK) return 0;
  return 0;
}

extern "C" int pa_paged_attention_decode_tree(const pa_decode_desc *d, const void *q, const void *k_pool,
                                              const void *v_pool, const int32_t *block_tables,
                                              const int32_t *context_lens, const int32_t *cu_nodes,
                                              const int32_t *parents, int max_tree_nodes, int total_nodes, void *out,
                                              void *workspace, size_t workspace_bytes, int32_t *err_flag,
                                              void *stream) {
  using namespace pa;
  const int vs = validate_tree(d, max_tree_nodes);
  if (vs != PA_OK) return vs;
  if (total_nodes < 0) return PA_ERR_INVALID;
  if (d->num_seqs == 0 || total_nodes == 0) return PA_OK;
  if (!q || !k_pool || !v_pool || !block_tables || !context_lens || !cu_nodes || !parents || !out)
    return PA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out)) return PA_ERR_INVALID;
  if (d->num_seqs > 65535 || d->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  TreeArgs a{};
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.k = static_cast<const __nv_bfloat16 *>(k_pool);
  a.v = static_cast<const __nv_bfloat16 *>(v_pool);
  a.bt = block_tables;
  a.ctx = context_lens;
  a.cu = cu_nodes;
  a.parents = parents;
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.err = err_flag;
  a.S = d->num_seqs;
  a.Hq = d->num_q_heads;
  a.Hkv = d->num_kv_heads;
  a.G = d->num_q_heads / d->num_kv_heads;
  a.B = d->block_size;
  a.num_blocks = d->num_blocks;
  a.max_blocks = d->max_blocks_per_seq;
  a.max_ctx = d->max_context_len;
  a.max_nodes = max_tree_nodes;
  a.total = total_nodes;
  a.scale_log2 = d->scale * 1.4426950408889634f;
  const dim3 grid(max_tree_nodes, d->num_kv_heads, d->num_seqs);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d->head_dim == 128)
    tree_kernel<128><<<grid, kTrWarps * 32, 0, st>>>(a);
  else
    tree_kernel<64><<<grid, kTrWarps * 32, 0, st>>>(a);
  return launch_status(cudaGetLastError());
}
