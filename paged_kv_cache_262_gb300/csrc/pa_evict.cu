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

// grid (kv head, sequence).  A row of weights that fits is held in shared
// memory as it is (keys are made of it as they are looked at), so that what is
// kept leaves straight from there, in place or not; a longer one is read again
// for each pass, and its kept weights move by stretches, read before they are
// written.
template <int NT>
__global__ void __launch_bounds__(NT) evict_select_kernel(const EvictArgs a) {
  extern __shared__ float sw[];
  __shared__ SelectSmem<NT> sm;
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
    for (int t = tid; t < s; t += NT) dup |= __ldg(a.rows + t) == row;
    if (__syncthreads_or(dup)) bits |= PA_DEVERR_ROW;
  }
  const int n = bits ? 0 : min(keep, ctx);
  if (h == 0 && tid == 0) {
    a.new_lens[s] = bits ? ctx : n;
    if (bits && a.err) atomicOr(a.err, bits);
  }
  for (int i = n + tid; i < a.max_keep; i += NT) kept[i] = -1;
  if (bits) return;
  const size_t wrow = ((size_t)row * a.Hkv + h) * a.max_tokens;
  const float *w = a.w_in + wrow;
  float *wo = a.w_out + wrow;
  if (n == ctx) {
    for (int i = tid; i < n; i += NT) kept[i] = i;
    if (wo != w)
      for (int i = tid; i < n; i += NT) wo[i] = w[i];
    return;
  }
  const int N = ctx - a.sink - a.recent, want = n - a.sink - a.recent;
  const bool in_smem = ctx <= a.smem_keys;
  if (in_smem) {
#pragma unroll 8
    for (int i = tid; i < ctx; i += NT) sw[i] = __ldcs(w + i);
    __syncthreads();
  }
  auto put = [&](int i, int j) {  // token j is kept, as number i
    kept[i] = j;
    if (in_smem) wo[i] = sw[j];
  };
  for (int i = tid; i < a.sink; i += NT) put(i, i);
  for (int i = tid; i < a.recent; i += NT) put(n - a.recent + i, ctx - a.recent + i);
  if (want > 0) {
    auto key = [&](int i) -> uint32_t { return order_key(in_smem ? sw[a.sink + i] : w[a.sink + i]); };
    const Kth<uint32_t> t = kth_largest<NT, uint32_t>(key, N, want, sm, tid);
    take_above<NT, uint32_t>(key, N, t.key, want - t.above, want, sm, tid,
                             [&](int pos, int i) { put(a.sink + pos, a.sink + i); });
  }
  if (in_smem) {
    for (int i = n + tid; i < ctx; i += NT) wo[i] = 0.f;
    return;
  }
  __syncthreads();
  for (int base = 0; base < ctx; base += NT) {
    const int i = base + tid;
    const float v = i < n ? w[min(max(kept[i], 0), ctx - 1)] : 0.f;
    __syncthreads();
    if (i < ctx) wo[i] = v;
  }
}

// Rows of K (even) or V (odd) of one (sequence, kv head), CPS 16-byte chunks
// of each: grid (2 * slices, kv head, sequence).  A stretch's rows are on
// their way while the one before is stored, and the list and table entries of
// the one after while both are: sources lie at or behind the stretch, so
// reading ahead of the stores changes nothing, and the barrier before the
// stores of a stretch ends its reads.
constexpr int kMvThreads = 256;
#ifndef PA_MV_UNROLL
#define PA_MV_UNROLL 4
#endif
#ifndef PA_MV_CPS
#define PA_MV_CPS 4
#endif
constexpr int kMvUnroll = PA_MV_UNROLL;

template <int D, int CPS>
__global__ void __launch_bounds__(kMvThreads) evict_move_kernel(const EvictArgs a) {
  constexpr int C = D / 8;
  constexpr int T = kMvThreads / CPS;  // tokens an access of the CTA covers
  constexpr int U = kMvUnroll;
  const int s = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  const int c = (blockIdx.x >> 1) * CPS + tid % CPS, t0 = tid / CPS;
  const int n = min(__ldg(a.new_lens + s), a.max_keep);
  const int32_t *kept = a.kept + ((size_t)s * a.Hkv + h) * a.max_keep;
  if (n <= 0 || __ldg(kept) < 0) return;
  uint4 *pool = (blockIdx.x & 1) ? a.vp : a.kp;
  const int32_t *bt = a.bt + (size_t)s * a.max_blocks, *dt = a.dst + (size_t)s * a.max_blocks;
  const int B = a.B, lb = B == 16 ? 4 : 5;
  int bad = 0;
  int j[U], sb[U], db[U];       // list and table entries of the stretch to load
  int64_t to[U], to_next[U];
  uint4 x[U], x_next[U];
  auto entries = [&](int base) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = base + u * T + t0;
      j[u] = i < n ? __ldg(kept + i) : -1;
      db[u] = i < n ? __ldg(dt + (i >> lb)) : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) sb[u] = j[u] >= 0 && (j[u] >> lb) < a.max_blocks ? __ldg(bt + (j[u] >> lb)) : -1;
  };
  auto load = [&](int base) {  // of the entries at hand
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = base + u * T + t0;
      to_next[u] = -1;
      if (i >= n) continue;
      if (sb[u] < 0 || sb[u] >= a.num_blocks || db[u] < 0 || db[u] >= a.num_blocks) {
        bad = 1;
      } else if (sb[u] != db[u] || ((i ^ j[u]) & (B - 1))) {
        to_next[u] = (((int64_t)db[u] * a.Hkv + h) * B + (i & (B - 1))) * C + c;
        x_next[u] = __ldcg(pool + (((int64_t)sb[u] * a.Hkv + h) * B + (j[u] & (B - 1))) * C + c);
      }
    }
  };
  entries(0);
  load(0);
  entries(T * U);
  for (int base = 0; base < n; base += T * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      to[u] = to_next[u];
      x[u] = x_next[u];
    }
    load(base + T * U);
    entries(base + 2 * T * U);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (to[u] >= 0) pool[to[u]] = x[u];
  }
  if (bad && a.err) atomicOr(a.err, PA_DEVERR_PAGE);
}

template <int D>
int launch_move(const EvictArgs &a, cudaStream_t st) {
  constexpr int CPS = PA_MV_CPS;
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
  // Short rows take small CTAs, several an SM.
  constexpr int kShort = 4096, kLong = 48 * 1024;
  a.smem_keys = std::min(d->max_context_len, kLong);
  const size_t smem = (size_t)a.smem_keys * 4;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->max_context_len <= kShort) {
    evict_select_kernel<256><<<dim3(a.Hkv, a.S), 256, smem, s>>>(a);
  } else {
    if (cudaFuncSetAttribute(evict_select_kernel<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLong * 4) !=
        cudaSuccess)
      return PA_ERR_CUDA;
    evict_select_kernel<1024><<<dim3(a.Hkv, a.S), 1024, smem, s>>>(a);
  }
  const int st = launch_status(cudaGetLastError());
  if (st != PA_OK) return st;
  return d->head_dim == 128 ? launch_move<128>(a, s) : launch_move<64>(a, s);
}
