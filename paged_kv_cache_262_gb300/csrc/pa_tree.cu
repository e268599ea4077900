// Verification of trees of drafted tokens and compaction of their accepted
// paths in the paged cache, for sm_103a.
//
// verify: every node's target is the largest of its logits, and a tree's path
// goes from node 0 to the child whose token is its parent's target, and on.
// commit: the path's K/V move up behind the context, slot c + i := slot
// c + path[i], in every layer.  Both belong to the decode phase of "Configuring
// vLLM and PagedAttention for High Throughput Enterprise LLM Serving" ("Memory
// Bottlenecks in Autoregressive LLM Inference") and to its block tables
// ("Architectural Foundations").
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_internal.h"
#include "pa_tree.cuh"
#include "pagedattn.h"

namespace pa {
namespace {

// A logit and its token in one word, the larger the better: the value's bits
// in its order (NaN above all, -0 as 0), then the lower token.
__device__ __forceinline__ unsigned long long rank_of(float x, int v) {
  const int b = __float_as_int(x + 0.f);
  const unsigned int o = x != x ? 0xffffffffu : (unsigned int)(b < 0 ? ~b : b ^ 0x80000000);
  return (unsigned long long)o << 32 | (unsigned int)~v;
}

struct VerifyArgs {
  const void *logits;
  int64_t stride;
  const int32_t *tokens, *parents, *cu;
  int32_t *targets, *path, *path_lens, *next;
  int32_t *err;
  int S, V, max_nodes, total;
};

constexpr int kVThreads = 256;

// grid (node, sequence): the node's target.
template <class T>
__global__ void __launch_bounds__(kVThreads) target_kernel(const VerifyArgs a) {
  const int i = blockIdx.x, s = blockIdx.y;
  const TreeRange r = tree_range(a.cu, s, a.total, a.max_nodes);
  if (r.bad || i >= r.count) return;
  const T *x = static_cast<const T *>(a.logits) + (size_t)(r.first + i) * a.stride;
  unsigned long long best = 0;
  for (int v = threadIdx.x; v < a.V; v += kVThreads) {
    const unsigned long long k = rank_of((float)x[v], v);
    best = k > best ? k : best;
  }
  __shared__ unsigned long long red[kVThreads];
  red[threadIdx.x] = best;
  __syncthreads();
  for (int o = kVThreads / 2; o > 0; o >>= 1) {
    if (threadIdx.x < o && red[threadIdx.x + o] > red[threadIdx.x]) red[threadIdx.x] = red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) a.targets[r.first + i] = (int32_t)~(unsigned int)red[0];
}

// One warp a sequence: the walk.
__global__ void __launch_bounds__(32) walk_kernel(const VerifyArgs a) {
  const int s = blockIdx.x, lane = threadIdx.x;
  const TreeRange r = tree_range(a.cu, s, a.total, a.max_nodes);
  if (r.bad && lane == 0 && a.err) atomicOr(a.err, PA_DEVERR_TREE);
  const int T = r.bad ? 0 : r.count;
  int32_t *path = a.path + (size_t)s * a.max_nodes;
  bool bad = false;
  for (int i = lane; i < T; i += 32) bad |= !good_parent(i, a.parents[r.first + i]);
  if (bad && a.err) atomicOr(a.err, PA_DEVERR_TREE);
  int n = 0, next = -1;
  int node = T > 0 && a.parents[r.first] == -1 ? 0 : -1;
  while (node >= 0) {
    if (lane == 0) path[n] = node;
    ++n;
    next = a.targets[r.first + node];
    int found = -1;
    for (int base = node + 1; base < T && found < 0; base += 32) {
      const int i = base + lane;
      const unsigned fits = __ballot_sync(
          0xffffffffu, i < T && a.parents[r.first + i] == node && a.tokens[r.first + i] == next);
      if (fits) found = base + __ffs(fits) - 1;
    }
    node = found;
  }
  for (int i = n + lane; i < a.max_nodes; i += 32) path[i] = -1;
  if (lane == 0) {
    a.path_lens[s] = n;
    a.next[s] = next;
  }
}

constexpr int kCommitLayers = 128;  // layers per launch (kernel-parameter space)

struct CommitArgs {
  uint4 *k[kCommitLayers], *v[kCommitLayers];
  const int32_t *bt, *ctx, *path, *path_lens;
  int32_t *new_lens;
  int32_t *err;
  int Hkv, B, C, num_blocks, max_blocks, max_ctx, max_path;
  int first;  // the launch that reports and writes new_lens
};

constexpr int kCThreads = 128;

// grid (sequence, layer, K|V).  path[i] >= i, so a row's source lies at or
// behind its destination, and rows moved in order never meet one that is
// still to be read.
__global__ void __launch_bounds__(kCThreads) commit_kernel(const __grid_constant__ CommitArgs a) {
  __shared__ int src[PA_MAX_TREE_NODES];
  const int s = blockIdx.x, tid = threadIdx.x;
  const bool told = a.first && blockIdx.y == 0 && blockIdx.z == 0 && tid == 0;
  const int c = __ldg(a.ctx + s), n = __ldg(a.path_lens + s);
  int why = c < 0 || n < 0 || n > a.max_path ? PA_DEVERR_CTX : 0;
  const int limit = min(a.max_ctx, a.max_blocks * a.B);
  const int32_t *path = a.path + (size_t)s * a.max_path;
  bool bad = false;
  if (!why)
    for (int i = tid; i < n; i += kCThreads) {
      const int p = __ldg(path + i), before = i > 0 ? __ldg(path + i - 1) : -1;
      src[i] = p;
      bad |= p <= before || p < 0 || p >= limit - c;
    }
  if (__syncthreads_or(bad)) why = PA_DEVERR_TREE;
  if (told) {
    a.new_lens[s] = why ? c : c + n;
    if (why && a.err) atomicOr(a.err, why);
  }
  if (why) return;
  uint4 *pool = blockIdx.z ? a.v[blockIdx.y] : a.k[blockIdx.y];
  for (int x = tid; x < a.Hkv * a.C; x += kCThreads) {
    const int h = x / a.C, ch = x - h * a.C;
    for (int i = 0; i < n; ++i) {
      if (src[i] == i) continue;
      const int from = c + src[i], to = c + i;
      const int fp = __ldg(a.bt + (size_t)s * a.max_blocks + from / a.B);
      const int tp = __ldg(a.bt + (size_t)s * a.max_blocks + to / a.B);
      if (fp < 0 || fp >= a.num_blocks || tp < 0 || tp >= a.num_blocks) {
        if (a.err) atomicOr(a.err, PA_DEVERR_PAGE);
        continue;
      }
      pool[(((size_t)tp * a.Hkv + h) * a.B + to % a.B) * a.C + ch] =
          pool[(((size_t)fp * a.Hkv + h) * a.B + from % a.B) * a.C + ch];
    }
  }
}

bool valid_verify(int num_seqs, int max_nodes, int vocab) { return num_seqs >= 0 && max_nodes > 0 && vocab > 0; }

}  // namespace
}  // namespace pa

extern "C" size_t pa_verify_tree_workspace_bytes(int num_seqs, int max_tree_nodes, int vocab_size) {
  return 0;
}

extern "C" int pa_verify_tree(const void *logits, int logits_type, int64_t logits_stride, int vocab_size,
                              const int32_t *tokens, const int32_t *parents, const int32_t *cu_nodes, int num_seqs,
                              int max_tree_nodes, int total_nodes, int32_t *targets, int32_t *path,
                              int32_t *path_lens, int32_t *next_tokens, void *workspace, size_t workspace_bytes,
                              int32_t *err_flag, void *stream) {
  using namespace pa;
  if (!valid_verify(num_seqs, max_tree_nodes, vocab_size) || total_nodes < 0 || logits_stride < vocab_size ||
      (logits_type != PA_LOGITS_BF16 && logits_type != PA_LOGITS_F32))
    return PA_ERR_INVALID;
  if (max_tree_nodes > PA_MAX_TREE_NODES || num_seqs > 65535) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  if (!cu_nodes || !path || !path_lens || !next_tokens ||
      (total_nodes > 0 && (!logits || !tokens || !parents || !targets)))
    return PA_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(logits) % (logits_type == PA_LOGITS_BF16 ? 2 : 4)) return PA_ERR_INVALID;
  VerifyArgs a{};
  a.logits = logits;
  a.stride = logits_stride;
  a.tokens = tokens;
  a.parents = parents;
  a.cu = cu_nodes;
  a.targets = targets;
  a.path = path;
  a.path_lens = path_lens;
  a.next = next_tokens;
  a.err = err_flag;
  a.S = num_seqs;
  a.V = vocab_size;
  a.max_nodes = max_tree_nodes;
  a.total = total_nodes;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(max_tree_nodes, num_seqs);
  if (logits_type == PA_LOGITS_BF16)
    target_kernel<__nv_bfloat16><<<grid, kVThreads, 0, st>>>(a);
  else
    target_kernel<float><<<grid, kVThreads, 0, st>>>(a);
  walk_kernel<<<num_seqs, 32, 0, st>>>(a);
  return launch_status(cudaGetLastError());
}

extern "C" int pa_commit_tree(const pa_decode_desc *d, void *const *k_pools, void *const *v_pools, int num_layers,
                              const int32_t *block_tables, const int32_t *context_lens, const int32_t *path,
                              const int32_t *path_lens, int max_path_len, int32_t *new_lens, int32_t *err_flag,
                              void *stream) {
  using namespace pa;
  const int vs = validate_decode_desc(d);
  if (vs != PA_OK) return vs;
  if (num_layers <= 0 || num_layers > 256 || max_path_len <= 0 || !k_pools || !v_pools) return PA_ERR_INVALID;
  if (max_path_len > PA_MAX_TREE_NODES) return PA_ERR_UNSUPPORTED;
  for (int l = 0; l < num_layers; ++l)
    if (!k_pools[l] || !v_pools[l] || !aligned16(k_pools[l]) || !aligned16(v_pools[l])) return PA_ERR_INVALID;
  if (d->num_seqs == 0) return PA_OK;
  if (!block_tables || !context_lens || !path || !path_lens || !new_lens) return PA_ERR_INVALID;
  const size_t S = d->num_seqs;
  if (!apart(new_lens, S, context_lens, S) || !apart(new_lens, S, path_lens, S) ||
      !apart(new_lens, S, path, S * max_path_len) || !apart(new_lens, S, block_tables, S * d->max_blocks_per_seq))
    return PA_ERR_INVALID;
  CommitArgs a{};
  a.bt = block_tables;
  a.ctx = context_lens;
  a.path = path;
  a.path_lens = path_lens;
  a.new_lens = new_lens;
  a.err = err_flag;
  a.Hkv = d->num_kv_heads;
  a.B = d->block_size;
  a.C = d->head_dim / 8;
  a.num_blocks = d->num_blocks;
  a.max_blocks = d->max_blocks_per_seq;
  a.max_ctx = d->max_context_len;
  a.max_path = max_path_len;
  for (int l0 = 0; l0 < num_layers; l0 += kCommitLayers) {
    const int nl = std::min(kCommitLayers, num_layers - l0);
    for (int l = 0; l < nl; ++l) {
      a.k[l] = static_cast<uint4 *>(k_pools[l0 + l]);
      a.v[l] = static_cast<uint4 *>(v_pools[l0 + l]);
    }
    a.first = l0 == 0;
    commit_kernel<<<dim3(d->num_seqs, nl, 2), kCThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    const int st = launch_status(cudaGetLastError());
    if (st != PA_OK) return st;
  }
  return PA_OK;
}
