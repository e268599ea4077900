// Eviction from the paged KV cache by accumulated attention weight, sm_103a:
// every (sequence, kv head) keeps its first `sink` tokens, its last `recent`
// ones and, of the rest, those with the largest accumulated weight
// (pa_decode_weights.cu), up to the sequence's keep_len; their K and V rows
// move, in order, to the first slots of the sequence's (destination) blocks,
// and their weights to the front of the weight row.  Rotary position is part
// of the cached keys, so a kept token may sit in any slot.  What a cache costs
// in memory and in bytes per step grows with the context ("Configuring vLLM
// and PagedAttention for High Throughput Enterprise LLM Serving", "Memory
// Bottlenecks in Autoregressive LLM Inference"); this bounds both.
//
// Two kernels: one CTA a (sequence, kv head) selects and lists the kept
// tokens, then the rows move.  The list increases, so slot i receives a token
// from slot >= i: a CTA that walks the list in order, reads a stretch before it
// writes it, and shares its rows with no other CTA may move them in place.  The
// rows are therefore cut along d (K and V apart), not along the list.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_internal.h"
#include "pa_select.cuh"
#include "pagedattn.h"

namespace pa {
namespace {

struct EvictArgs {
  uint4 *kp, *vp;
  const int32_t *bt, *dst;
  const int32_t *ctx, *keep;
  const float *w_in;
  float *w_out;
  const int32_t *rows;
  int32_t *kept;      // [S][Hkv][max_keep]
  int32_t *new_lens;  // [S]
  int32_t *err;
  int S, Hkv, B, num_blocks, max_blocks, max_ctx, max_keep, sink, recent, num_rows, smem_keys;
  size_t max_tokens;
};

constexpr int kEvThreads = 1024;

// grid (kv head, sequence)
__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(const EvictArgs a) {
  extern __shared__ uint32_t skeys[];
  __shared__ SelectSmem<kEvThreads> sm;
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
  int32_t *kept = a.kept + ((size_t)s * a.Hkv + h) * a.max_keep;
  const int ctx = __ldg(a.ctx + s), keep = __ldg(a.keep + s);
  const int row = a.rows ? __ldg(a.rows + s) : s;
  int bits = 0;
  if (ctx <= 0 || ctx > a.max_blocks * a.B || ctx > a.max_ctx || keep <= 0 || keep > a.max_keep ||
      (keep < ctx && (long long)a.sink + a.recent > keep))
    bits |= PA_DEVERR_CTX;
  if (row < 0 || row >= a.num_rows) bits |= PA_DEVERR_ROW;
  if (a.rows && !bits) {  // a row that an earlier sequence names is that one's
    bool dup = false;
    for (int t = tid; t < s; t += kEvThreads) dup |= __ldg(a.rows + t) == row;
    if (__syncthreads_or(dup)) bits |= PA_DEVERR_ROW;
  }
  const int n = bits ? 0 : min(keep, ctx);
  if (h == 0 && tid == 0) {
    a.new_lens[s] = bits ? ctx : n;
    if (bits && a.err) atomicOr(a.err, bits);
  }
  for (int i = n + tid; i < a.max_keep; i += kEvThreads) kept[i] = -1;
  if (bits) return;
  const size_t wrow = ((size_t)row * a.Hkv + h) * a.max_tokens;
  const float *w = a.w_in + wrow;
  if (n == ctx) {
    for (int i = tid; i < n; i += kEvThreads) kept[i] = i;
  } else {
    for (int i = tid; i < a.sink; i += kEvThreads) kept[i] = i;
    for (int i = tid; i < a.recent; i += kEvThreads) kept[n - a.recent + i] = ctx - a.recent + i;
    const int N = ctx - a.sink - a.recent, want = n - a.sink - a.recent;
    if (want > 0) {
      const bool in_smem = N <= a.smem_keys;
      if (in_smem) {
        for (int i = tid; i < N; i += kEvThreads) skeys[i] = order_key(w[a.sink + i]);
        __syncthreads();
      }
      auto key = [&](int i) -> uint32_t { return in_smem ? skeys[i] : order_key(w[a.sink + i]); };
      const Kth<uint32_t> t = kth_largest<kEvThreads, uint32_t>(key, N, want, sm, tid);
      take_above<kEvThreads, uint32_t>(key, N, t.key, want - t.above, want, sm, tid,
                                       [&](int pos, int i) { kept[a.sink + pos] = a.sink + i; });
    }
  }
  // the weights, in place or not: a stretch is read before it is written, and
  // what is written was read (kept increases)
  __syncthreads();
  float *wo = a.w_out + wrow;
  for (int base = 0; base < ctx; base += kEvThreads) {
    const int i = base + tid;
    const float v = i < n ? w[min(max(kept[i], 0), ctx - 1)] : 0.f;
    __syncthreads();
    if (i < ctx) wo[i] = v;
  }
}

// Rows of K (even) or V (odd) of one (sequence, kv head), CPS 16-byte chunks
// of each: grid (2 * slices, kv head, sequence).
constexpr int kMvThreads = 256;
constexpr int kMvUnroll = 4;

template <int D, int CPS>
__global__ void __launch_bounds__(kMvThreads) evict_move_kernel(const EvictArgs a) {
  constexpr int C = D / 8;
  constexpr int T = kMvThreads / CPS;  // tokens an access of the CTA covers
  const int s = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  const int c = (blockIdx.x >> 1) * CPS + tid % CPS, t0 = tid / CPS;
  const int n = min(__ldg(a.new_lens + s), a.max_keep);
  const int32_t *kept = a.kept + ((size_t)s * a.Hkv + h) * a.max_keep;
  if (n <= 0 || __ldg(kept) < 0) return;
  uint4 *pool = (blockIdx.x & 1) ? a.vp : a.kp;
  const int32_t *bt = a.bt + (size_t)s * a.max_blocks, *dt = a.dst + (size_t)s * a.max_blocks;
  const int B = a.B;
  int bad = 0;
  for (int base = 0; base < n; base += T * kMvUnroll) {
    uint4 x[kMvUnroll];
    int64_t to[kMvUnroll];
#pragma unroll
    for (int u = 0; u < kMvUnroll; ++u) {
      const int i = base + u * T + t0;
      to[u] = -1;
      if (i < n) {
        const int j = __ldg(kept + i);
        const int sb = j >= 0 && j / B < a.max_blocks ? __ldg(bt + j / B) : -1, db = __ldg(dt + i / B);
        if (sb < 0 || sb >= a.num_blocks || db < 0 || db >= a.num_blocks) {
          bad = 1;
        } else if (sb != db || j % B != i % B) {
          to[u] = (((int64_t)db * a.Hkv + h) * B + i % B) * C + c;
          x[u] = __ldcg(pool + (((int64_t)sb * a.Hkv + h) * B + j % B) * C + c);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMvUnroll; ++u)
      if (to[u] >= 0) pool[to[u]] = x[u];
  }
  if (bad && a.err) atomicOr(a.err, PA_DEVERR_PAGE);
}

template <int D>
int launch_move(const EvictArgs &a, cudaStream_t st) {
  constexpr int CPS = 4;
  evict_move_kernel<D, CPS><<<dim3(2 * (D / 8) / CPS, a.Hkv, a.S), kMvThreads, 0, st>>>(a);
  return launch_status(cudaGetLastError());
}

}  // namespace
}  // namespace pa

extern "C" int pa_evict_tokens(const pa_decode_desc *d, void *k_pool, void *v_pool, const int32_t *block_tables,
                               const int32_t *dst_tables, const int32_t *context_lens, const int32_t *keep_lens,
                               int max_keep_len, int sink_tokens, int recent_tokens, const float *weights,
                               float *weights_out, const int32_t *weight_rows, int num_rows, int max_tokens,
                               int32_t *kept, int32_t *new_lens, int32_t *err_flag, void *stream) {
  using namespace pa;
  const int vs = validate_decode_desc(d);
  if (vs != PA_OK) return vs;
  if (max_keep_len <= 0 || sink_tokens < 0 || recent_tokens < 0 || num_rows < 0 ||
      max_tokens < d->max_context_len || (!weight_rows && num_rows < d->num_seqs))
    return PA_ERR_INVALID;
  if (d->num_seqs == 0) return PA_OK;
  if (!k_pool || !v_pool || !block_tables || !context_lens || !keep_lens || !weights || !weights_out || !kept ||
      !new_lens || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(weights) || !aligned16(weights_out))
    return PA_ERR_INVALID;
  if (d->num_seqs > 65535 || d->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  EvictArgs a{};
  a.kp = static_cast<uint4 *>(k_pool);
  a.vp = static_cast<uint4 *>(v_pool);
  a.bt = block_tables;
  a.dst = dst_tables ? dst_tables : block_tables;
  a.ctx = context_lens;
  a.keep = keep_lens;
  a.w_in = weights;
  a.w_out = weights_out;
  a.rows = weight_rows;
  a.kept = kept;
  a.new_lens = new_lens;
  a.err = err_flag;
  a.S = d->num_seqs;
  a.Hkv = d->num_kv_heads;
  a.B = d->block_size;
  a.num_blocks = d->num_blocks;
  a.max_blocks = d->max_blocks_per_seq;
  a.max_ctx = d->max_context_len;
  a.max_keep = max_keep_len;
  a.sink = sink_tokens;
  a.recent = recent_tokens;
  a.num_rows = num_rows;
  a.max_tokens = (size_t)max_tokens;
  a.smem_keys = std::min(d->max_context_len, 48 * 1024);
  const size_t smem = (size_t)a.smem_keys * 4;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(48 * 1024 * 4)) !=
      cudaSuccess)
    return PA_ERR_CUDA;
  evict_select_kernel<<<dim3(a.Hkv, a.S), kEvThreads, smem, s>>>(a);
  const int st = launch_status(cudaGetLastError());
  if (st != PA_OK) return st;
  return d->head_dim == 128 ? launch_move<128>(a, s) : launch_move<64>(a, s);
}
