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
//
// Nothing is computed: the floor is the bytes, 8 D a kept token and kv head for
// K and V in and out, 8 a token for the weights.  At 8 x 32768 tokens kept to
// 16384 (8 kv heads, D 128; 1.09 GB) both take 196 us, 5.6 TB/s: 23 the
// selection, whose instructions bind (64 rows on 64 SMs; a cluster of CTAs a
// row measured the same), 172 the rows, 6.2 TB/s.  64 sequences of up to 2048
// tokens kept to 512: 51 us, 5.0 TB/s.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_internal.h"
#include "pa_ptx.cuh"
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

// Weights that nothing has written yet in this kernel: the compiler may order
// these loads as it likes, and so has several on their way.
__device__ __forceinline__ float4 load_weights(const float *p) {
  float4 x;
  asm("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "l"(p));
  return x;
}
__device__ __forceinline__ float load_weight(const float *p) {
  float x;
  asm("ld.global.f32 %0, [%1];" : "=f"(x) : "l"(p));
  return x;
}

// grid (kv head, sequence).  A row of weights that fits is held in shared
// memory as ordered keys, which give the weights back (NaN and -0 as the usual
// NaN and +0), so that what is kept leaves straight from there, in place or
// not; a longer one is read again for each pass, and its kept weights move by
// stretches, read before they are written.  SMEM: every row fits.
template <int NT, bool SMEM>
__global__ void __launch_bounds__(NT) evict_select_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint32_t skeys[];
  __shared__ SelectSmem<NT> sm;
  grid_wait();
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
  // keys of the tokens that compete, N of them behind the sinks
  const int N = ctx - a.sink - a.recent, want = n - a.sink - a.recent;
  const float *wc = w + a.sink;
  const bool in_smem = SMEM || N <= a.smem_keys;
  uint32_t least = ~0u, most = 0u;
  auto look = [&](int i, uint32_t k) {
    if (in_smem) skeys[i] = k;
    least = min(least, k);
    most = max(most, k);
  };
  if (want > 0) {
    const int head = min(N, (int)(-(reinterpret_cast<uintptr_t>(wc) >> 2) & 3));  // up to a 16-byte boundary
    if (tid < head) look(tid, order_key(wc[tid]));
    const float4 *wv = reinterpret_cast<const float4 *>(wc + head);
    const int nv = (N - head) / 4;
    for (int base = 0; base < nv; base += 8 * NT) {
      float4 x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (base + u * NT + tid < nv) x[u] = __ldcs(wv + base + u * NT + tid);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = base + u * NT + tid;
        if (i >= nv) break;
        const uint4 k = make_uint4(order_key(x[u].x), order_key(x[u].y), order_key(x[u].z), order_key(x[u].w));
        least = min(min(least, min(k.x, k.y)), min(k.z, k.w));
        most = max(max(most, max(k.x, k.y)), max(k.z, k.w));
        if (!in_smem) continue;
        uint32_t *to = skeys + head + 4 * i;
        if (head == 0)
          *reinterpret_cast<uint4 *>(to) = k;
        else
          to[0] = k.x, to[1] = k.y, to[2] = k.z, to[3] = k.w;
      }
    }
    const int i = head + 4 * nv + tid;
    if (i < N) look(i, order_key(wc[i]));
  }
  // the ends: sinks stay where they are, recent tokens are read before any write
  constexpr int kEnd = 4;
  float tail[kEnd];
#pragma unroll
  for (int e = 0; e < kEnd; ++e)
    if (e * NT + tid < a.recent) tail[e] = w[ctx - a.recent + e * NT + tid];
  __syncthreads();
  for (int i = tid; i < a.sink; i += NT) {
    kept[i] = i;
    if (wo != w) wo[i] = w[i];
  }
  for (int i = tid; i < a.recent; i += NT) kept[n - a.recent + i] = ctx - a.recent + i;
  if (want > 0) {
    // Not held: four weights a load, from a 16-byte boundary on; the `lead` ones
    // before the first get key 0, which is below every weight's.
    const int lead = in_smem ? 0 : (int)(reinterpret_cast<uintptr_t>(wc) >> 2) & 3;
    const float *wa = wc - lead;
    const int n_keys = N + lead;
    auto key4 = [&](int i) {
      if (in_smem) return keys4(*reinterpret_cast<const uint4 *>(skeys + i));
      Keys4<uint32_t> k;
      if (i + 4 <= n_keys) {
        const float4 x = load_weights(wa + i);
        k = Keys4<uint32_t>{{order_key(x.x), order_key(x.y), order_key(x.z), order_key(x.w)}};
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) k.v[e] = i + e < n_keys ? order_key(load_weight(wa + i + e)) : 0u;
      }
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (i + e < lead) k.v[e] = 0u;
      return k;
    };
    auto key1 = [&](int i) { return in_smem ? skeys[i] : i < lead ? 0u : order_key(load_weight(wa + i)); };
    const Kth<uint32_t> t = kth_largest<NT, uint32_t>(key4, n_keys, want, sm, tid, least, most);
    take_above<NT, uint32_t>(key4, key1, n_keys, t.key, want - t.above, want, sm, tid,
                             [&](int pos, int i, uint32_t k) {
                               kept[a.sink + pos] = a.sink + i - lead;
                               if (in_smem) wo[a.sink + pos] = key_value(k);
                             });
  }
  if (in_smem && a.recent <= kEnd * NT) {
#pragma unroll
    for (int e = 0; e < kEnd; ++e)
      if (e * NT + tid < a.recent) wo[n - a.recent + e * NT + tid] = tail[e];
    for (int i = n + tid; i < ctx; i += NT) wo[i] = 0.f;
    return;
  }
  __syncthreads();
  // by stretches; where the competing ones have gone already, the recent ones
  const int from = in_smem ? n - a.recent : 0;
  constexpr int kBatch = 8;
  for (int base = from; base < ctx; base += kBatch * NT) {
    float v[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int i = base + e * NT + tid;
      v[e] = i < n ? w[min(max(kept[i], 0), ctx - 1)] : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      if (base + e * NT + tid < ctx) wo[base + e * NT + tid] = v[e];
  }
}

// Rows of K (even) or V (odd) of one (sequence, kv head), RB bytes of each:
// grid (2 * slices, kv head, sequence).  The rows go through a ring of stages
// in shared memory by asynchronous copies, a 16-byte piece a thread and stage;
// a thread stores the pieces that it loaded.  A stage is stored when every
// thread's copies of it, and of all before it, have landed; the later ones on
// their way read at or behind their own slots, which no earlier stage writes.
constexpr int kMvThreads = 256;
constexpr int kMvPieces = 4;  // pieces of a thread in a stage

__device__ __forceinline__ void copy16_async(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// ST stages; IX rows of list and table entries, ahead and behind, looked up IR
// rows a thread at a time.
template <int ST, int IX>
struct MoveSmem {
  uint4 ring[ST][kMvPieces][kMvThreads];
  int32_t src[IX], dst[IX];  // pool rows; dst -1: the row stays where it is
};

template <int D, int RB, int ST, int IX, int IR>
__global__ void __launch_bounds__(kMvThreads) evict_move_kernel(const EvictArgs a) {
  constexpr int C = D / 8;              // 16-byte pieces of a row
  constexpr int P = RB / 16;            // of which a CTA moves
  constexpr int A = kMvThreads / P;     // rows of one piece a thread
  constexpr int T = A * kMvPieces;      // rows of a stage
  constexpr int IG = IR * kMvThreads;   // rows of an index group
  constexpr int GS = IG / T;            // stages it covers
  static_assert(T <= IG && IG % T == 0, "whole stages to an index group");
  static_assert(ST * T + 3 * IG <= IX, "the index ring holds what is in flight");
  extern __shared__ __align__(16) uint8_t smem_raw[];
  auto &sm = *reinterpret_cast<MoveSmem<ST, IX> *>(smem_raw);
  const int s = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  grid_wait();
  // (The kernel before writes these; of a refused sequence it is the context, which
  // may be past the table.)
  const int n = min(min(__ldcg(a.new_lens + s), a.max_keep), a.max_blocks * a.B);
  const int32_t *kept = a.kept + ((size_t)s * a.Hkv + h) * a.max_keep;
  const int32_t *bt = a.bt + (size_t)s * a.max_blocks, *dt = a.dst + (size_t)s * a.max_blocks;
  const int B = a.B, lb = B == 16 ? 4 : 5;
  uint4 *pool = ((blockIdx.x & 1) ? a.vp : a.kp) + (blockIdx.x >> 1) * P + tid % P;
  int bad = 0;

  // index groups: list entry, then the source block's table entry, then the
  // rows into shared memory, each a group ahead of the next
  int g1 = 0, g2 = 0, j1[IR], s1[IR], d1[IR], j2[IR], d2[IR];
  auto step_list = [&](int g) {
    g2 = g;
#pragma unroll
    for (int r = 0; r < IR; ++r) {
      const int i = g * IG + r * kMvThreads + tid;
      j2[r] = i < n ? __ldcg(kept + i) : -1;
      d2[r] = i < n ? __ldg(dt + (i >> lb)) : -1;
    }
  };
  auto step_table = [&]() {
    g1 = g2;
#pragma unroll
    for (int r = 0; r < IR; ++r) {
      j1[r] = j2[r], d1[r] = d2[r];
      s1[r] = j1[r] >= 0 && (j1[r] >> lb) < a.max_blocks ? __ldg(bt + (j1[r] >> lb)) : -1;
    }
  };
  auto step_rows = [&]() {
#pragma unroll
    for (int r = 0; r < IR; ++r) {
      const int i = g1 * IG + r * kMvThreads + tid;
      int32_t from = 0, to = -1;
      if (j1[r] >= 0) {
        if (s1[r] < 0 || s1[r] >= a.num_blocks || d1[r] < 0 || d1[r] >= a.num_blocks) {
          bad = 1;
        } else {
          from = (s1[r] * a.Hkv + h) * B + (j1[r] & (B - 1));
          const int32_t at = (d1[r] * a.Hkv + h) * B + (i & (B - 1));
          to = at == from ? -1 : at;
        }
      }
      sm.src[i % IX] = from;
      sm.dst[i % IX] = to;
    }
  };
  const uint32_t ring = smem_u32(&sm.ring[0][0][tid]);
  const int t0 = tid / P;
  auto load = [&](int st) {  // one group of copies, empty past the end
#pragma unroll
    for (int u = 0; u < kMvPieces; ++u) {
      const int i = st * T + u * A + t0;
      if (i < n && sm.dst[i % IX] >= 0)
        copy16_async(ring + ((st % ST) * kMvPieces + u) * (kMvThreads * 16),
                     pool + (int64_t)sm.src[i % IX] * C);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  step_list(0);
  if (n <= 0 || __ldcg(kept) < 0) return;  // a refused sequence (the same for the whole CTA)
  step_table();
  step_list(1);
  step_rows();
  step_table();
  step_list(2);
  __syncthreads();
  const int nst = (n + T - 1) / T;
  int made = 1;  // index groups in shared memory
#pragma unroll 1
  for (int st = 0; st < ST - 1; ++st) {
    if (st == made * GS) {
      step_rows();
      step_table();
      step_list(++made + 1);
      __syncthreads();
    }
    load(st);
  }
#pragma unroll 1
  for (int st = 0; st < nst; ++st) {
    const int ahead = st + ST - 1;
    if (ahead >= made * GS - 1) {  // read behind the barrier
      step_rows();
      step_table();
      step_list(++made + 1);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(ST - 2) : "memory");
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMvPieces; ++u) {
      const int i = st * T + u * A + t0;
      const int32_t to = i < n ? sm.dst[i % IX] : -1;
      if (to >= 0) pool[(int64_t)to * C] = sm.ring[st % ST][u][tid];
    }
    load(ahead);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (bad && a.err) atomicOr(a.err, PA_DEVERR_PAGE);
}

template <int D, int RB, int ST, int IX, int IR>
int launch_move_rows(const EvictArgs &a, cudaStream_t st) {
  using Smem = MoveSmem<ST, IX>;
  auto kern = evict_move_kernel<D, RB, ST, IX, IR>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem)) != cudaSuccess)
    return PA_ERR_CUDA;
  return launch_dependent(kern, dim3(2 * (D * 2 / RB), a.Hkv, a.S), kMvThreads, sizeof(Smem), 1, st, a);
}

// Whole rows where that gives three CTAs to two SMs, else parts of 128 or 64
// bytes; a CTA with an SM to itself takes more stages and larger index groups,
// and where parts of 64 bytes leave half the SMs idle, parts of a sector.  (us
// at 16384 of 32768 tokens, 8 kv heads: 8 sequences 194 by 128 bytes, 210 by
// 256; 1 sequence 60 by 32 bytes, 73 by 64.)  The selection does not let it start
// early: CTAs that start while the selection still holds some SMs pile up on the
// others (205 us instead of 194).
template <int D>
int launch_move(const EvictArgs &a, int sms, cudaStream_t st) {
  const int64_t units = 2ll * a.Hkv * a.S;
  if constexpr (D == 128)
    if (2 * units >= 3ll * sms) return launch_move_rows<D, 256, 3, 2048, 1>(a, st);
  if (2 * units * (D / 64) >= 3ll * sms) return launch_move_rows<D, 128, 3, 2048, 1>(a, st);
  const int64_t ctas = units * (D / 32);
  if (ctas > sms) return launch_move_rows<D, 64, 3, 2048, 1>(a, st);
  if (2 * ctas > sms) return launch_move_rows<D, 64, 4, 8192, 8>(a, st);
  return launch_move_rows<D, 32, 4, 8192, 8>(a, st);
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
      !new_lens || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(weights) || !aligned16(weights_out) ||
      !same_or_apart(weights, weights_out, num_rows, d->num_kv_heads, max_tokens))
    return PA_ERR_INVALID;
  // One kv head's CTA writes what the others' may not have read yet.
  const size_t S = d->num_seqs, tables = S * d->max_blocks_per_seq, list = S * d->num_kv_heads * max_keep_len;
  const struct {
    const int32_t *p;
    size_t n;
  } read[] = {{context_lens, S}, {keep_lens, S}, {weight_rows, S}, {block_tables, tables}, {dst_tables, tables}};
  for (const auto &r : read)
    if (!apart(new_lens, S, r.p, r.n) || !apart(kept, list, r.p, r.n)) return PA_ERR_INVALID;
  if (!apart(new_lens, S, kept, list)) return PA_ERR_INVALID;
  if (d->num_seqs > 65535 || d->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  const int sms = current_sm_count();
  if (sms <= 0) return PA_ERR_CUDA;
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
  const size_t smem = (size_t)((a.smem_keys + 3) & ~3) * 4;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(a.Hkv, a.S);
  int st;
  if (d->max_context_len <= kShort) {
    st = launch_dependent(evict_select_kernel<256, true>, grid, 256, smem, 1, s, a);
  } else {
    auto kern = d->max_context_len <= kLong ? evict_select_kernel<1024, true> : evict_select_kernel<1024, false>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kLong * 4) != cudaSuccess)
      return PA_ERR_CUDA;
    st = launch_dependent(kern, grid, 1024, smem, 1, s, a);
  }
  if (st != PA_OK) return st;
  return d->head_dim == 128 ? launch_move<128>(a, sms, s) : launch_move<64>(a, sms, s);
}
