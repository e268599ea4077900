// Paged decode attention that also sums every key's attention weight, for
// sm_103a: beside out = sum_j p_j v_j (pa_decode.cu), each cached token's
//   W[row][h][j] += sum over the kv head's query heads g of p_gj,
//   p_gj = 2^(x_gj - M_g) / L_g,  x = scale log2(e) q.k,
// the accumulated attention weight by which tokens are evicted (pa_evict.cu)
// -- the KV cache growing with the context is the bottleneck of "Configuring
// vLLM and PagedAttention for High Throughput Enterprise LLM Serving"
// ("Memory Bottlenecks in Autoregressive LLM Inference").
//
// p needs the row's final maximum and sum, which exist only once the whole
// context has been read.  Reading K again would cost half of the call once
// more; instead the decode unit (pa_decode_body.cuh) leaves its logits, 4 G
// bytes a (token, kv head) against the 4 D bytes of its K and V, and a second
// kernel turns them into weights.  The cache streams past L2 (evict first)
// while the logits are kept there (evict last) and let go as they are read.
//
// Where a CTA's own logits are few it adds their weights itself at its end, in
// the one launch.
//
// 8 x 32768 tokens, 64 query and 8 kv heads of 128 (1.09 GB): 182 us, 6.0 TB/s,
// 167 the first kernel (67 MB of logits written, 7 MB of them reach HBM; without
// the hint 204 us in all) and the rest the second, which starts while the first
// runs and has the old sums loaded when it ends.  64 sequences of 128 .. 2048
// tokens: 49 us, 6.1 TB/s.  Four sequences of up to 100: 4.4 us in a graph, the
// launch, and 5-6 a call from Python, the host's.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "pa_decode_body.cuh"
#include "pa_internal.h"
#include "pagedattn.h"

namespace pa {
namespace {

template <int D, int B, int NT, int NST, bool CL>
__global__ void __launch_bounds__(128)
    decode_logits_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const DecodeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  grid_wait();
  grid_launch_dependents();
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int lin = (blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
  decode_unit<D, B, NT, 4, NST, false, false, false, D == 128, false, true, CL>(&tmK, &tmV, a, lin, threadIdx.x, smem,
                                                                                0);
}

struct WeightArgs {
  const float *logits;    // [S][Hkv][max_ctx][G]
  const float2 *stats;    // [S][Hq]
  const int32_t *ctx;
  const int32_t *rows;    // [S] or null: row s
  const float *w_in;      // [num_rows][Hkv][max_tokens]
  float *w_out;
  int32_t *err;
  int S, Hkv, G, num_rows, max_ctx, max_tokens_table;
  size_t max_tokens;
};

constexpr int kWThreads = 128;
constexpr int kWPer = 4;  // tokens of a thread
constexpr int kWTokens = kWThreads * kWPer;

// grid (token chunk, kv head, sequence).  Sequences that name the same row
// are summed by the first of them, in sequence order, so that a row has one
// writer and its sums one order.  A token's G logits lie together: V of them
// a load (V divides G), one load of each of the thread's tokens in flight.
template <int V>
__global__ void __launch_bounds__(kWThreads) weights_kernel(const WeightArgs a) {
  using Vec = typename FloatVec<V>::type;
  extern __shared__ uint32_t members[];  // bit s: sequence s names this CTA's row
  __shared__ float2 sst[2][16];          // statistics of the query heads, of this sequence and the next
  const int s = blockIdx.z, h = blockIdx.y, j0 = blockIdx.x * kWTokens, tid = threadIdx.x;
  const int row = a.rows ? __ldg(a.rows + s) : s;
  const bool in_range = row >= 0 && row < a.num_rows;
  bool mine = in_range;
  if (a.rows && in_range) {
    for (int base = 0; base < a.S; base += kWThreads) {
      const int t = base + tid;
      const bool same = t < a.S && __ldg(a.rows + t) == row;
      mine &= !(same && t < s);
      const unsigned int b = __ballot_sync(0xffffffffu, same);
      if ((tid & 31) == 0) members[t >> 5] = b;
    }
    mine = __syncthreads_and(mine);
  } else if (mine) {
    mine = __ldg(a.ctx + s) > j0;
  }
  const size_t wrow = ((size_t)(mine ? row : 0) * a.Hkv + h) * a.max_tokens;
  float w[kWPer];  // on their way while the logits are still written
#pragma unroll
  for (int i = 0; i < kWPer; ++i) {
    const int j = j0 + i * kWThreads + tid;
    w[i] = mine && j < a.max_ctx ? a.w_in[wrow + j] : 0.f;
  }
  grid_wait();  // the logits are complete
  if (!in_range && a.err && tid == 0 && h == 0 && blockIdx.x == 0) atomicOr(a.err, PA_DEVERR_ROW);
  if (!mine) return;
  float acc[kWPer];
  bool any[kWPer];
#pragma unroll
  for (int i = 0; i < kWPer; ++i) acc[i] = 0.f, any[i] = false;
  const uint64_t done = policy_evict_first();  // the logits leave L2 first once read
  const int words = a.rows ? (a.S + 31) / 32 : 1;
  int flip = 0;
  for (int w = 0; w < words; ++w) {
    uint32_t left = a.rows ? members[w] : 1u;
    while (left) {
      const int t = a.rows ? w * 32 + __ffs(left) - 1 : s;
      left &= left - 1;
      const int ctx = __ldg(a.ctx + t);
      if (ctx <= j0 || ctx > a.max_ctx || ctx > a.max_tokens_table) continue;
      if (tid < a.G) sst[flip][tid] = __ldcg(a.stats + ((size_t)t * a.Hkv + h) * a.G + tid);
      __syncthreads();  // (two buffers: who is behind still reads the other)
      const float2 *st = sst[flip];
      flip ^= 1;
      const Vec *lg = reinterpret_cast<const Vec *>(a.logits + ((size_t)t * a.Hkv + h) * a.max_ctx * a.G);
      float sum[kWPer];
#pragma unroll
      for (int i = 0; i < kWPer; ++i) sum[i] = 0.f;
#pragma unroll 2
      for (int g = 0; g < a.G; g += V) {
        Vec x[kWPer];
#pragma unroll
        for (int i = 0; i < kWPer; ++i) {
          const int j = j0 + i * kWThreads + tid;
          if (j < ctx) x[i] = load_hint(lg + ((size_t)j * a.G + g) / V, done);
        }
#pragma unroll
        for (int i = 0; i < kWPer; ++i)
#pragma unroll
          for (int e = 0; e < V; ++e)
            sum[i] += ex2_ftz(reinterpret_cast<const float *>(&x[i])[e] - st[g + e].x) * st[g + e].y;
      }
#pragma unroll
      for (int i = 0; i < kWPer; ++i)
        if (j0 + i * kWThreads + tid < ctx) {
          acc[i] += sum[i];
          any[i] = true;
        }
    }
  }
#pragma unroll
  for (int i = 0; i < kWPer; ++i) {
    const int j = j0 + i * kWThreads + tid;
    if (any[i]) a.w_out[wrow + j] = w[i] + acc[i];
  }
}

struct WeightPlan {
  DecodePlan split;
  size_t stats = 0, logits = 0;
  size_t total() const { return split.total() + stats + logits; }
};

WeightPlan make_plan(const pa_decode_desc *d, int sms) {
  WeightPlan p;
  p.split = make_cluster_plan(d, sms);
  auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
  const size_t G = d->num_q_heads / d->num_kv_heads, units = (size_t)d->num_seqs * d->num_kv_heads;
  p.stats = up(units * G * sizeof(float2));
  p.logits = up(units * G * (size_t)d->max_context_len * sizeof(float));
  return p;
}

template <int D, int B, int NT, int NST>
int launch_logits(const pa_decode_desc *d, const CUtensorMap &tk, const CUtensorMap &tv, const DecodeArgs &a,
                  cudaStream_t st) {
  return launch_parts(decode_logits_kernel<D, B, NT, NST, false>, decode_logits_kernel<D, B, NT, NST, true>,
                      DecodeSmem<D, B, 4, NST>::kAlloc, d, 128, tk, tv, a, st);
}

// Slots of a warp as in the plain decode: 16-token pages two when the units fit
// one wave, else three; 32-token pages one.
template <int D, int B>
int dispatch_logits(const pa_decode_desc *d, const CUtensorMap &tk, const CUtensorMap &tv, const DecodeArgs &a,
                    int sms, cudaStream_t st) {
  if constexpr (B == 16) {
    if (a.G <= 8 && (long long)a.max_parts * a.Hkv * a.S <= 2ll * sms)
      return launch_logits<D, B, 1, 2>(d, tk, tv, a, st);
    return a.G <= 8 ? launch_logits<D, B, 1, 3>(d, tk, tv, a, st) : launch_logits<D, B, 2, 3>(d, tk, tv, a, st);
  } else {
    return a.G <= 8 ? launch_logits<D, B, 1, 1>(d, tk, tv, a, st) : launch_logits<D, B, 2, 1>(d, tk, tv, a, st);
  }
}

}  // namespace
}  // namespace pa

extern "C" size_t pa_decode_weights_workspace_bytes(const pa_decode_desc *d) {
  using namespace pa;
  if (validate_decode_desc(d) != PA_OK) return 0;
  return make_plan(d, current_sm_count()).total();
}

extern "C" int pa_paged_attention_decode_weights(const pa_decode_desc *d, const void *q, const void *k_pool,
                                                 const void *v_pool, const int32_t *block_tables,
                                                 const int32_t *context_lens, const float *weights, float *weights_out,
                                                 const int32_t *weight_rows, int num_rows, int max_tokens, void *out,
                                                 void *workspace, size_t workspace_bytes, int32_t *err_flag,
                                                 void *stream) {
  using namespace pa;
  const int vs = validate_decode_desc(d);
  if (vs != PA_OK) return vs;
  if (num_rows < 0 || max_tokens < d->max_context_len || (!weight_rows && num_rows < d->num_seqs))
    return PA_ERR_INVALID;
  if (d->num_seqs == 0) return PA_OK;
  if (!q || !k_pool || !v_pool || !block_tables || !context_lens || !weights || !weights_out || !out)
    return PA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out) || !aligned16(weights) ||
      !aligned16(weights_out) || !same_or_apart(weights, weights_out, num_rows, d->num_kv_heads, max_tokens))
    return PA_ERR_INVALID;
  if (d->num_seqs > 65535 || d->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  const int sms = current_sm_count();
  if (sms <= 0) return PA_ERR_CUDA;
  const WeightPlan plan = make_plan(d, sms);
  if (!workspace || workspace_bytes < plan.total() || !aligned16(workspace)) return PA_ERR_WORKSPACE;
  CUtensorMap tk, tv;
  if (!encode_kv_pages(d, k_pool, &tk) || !encode_kv_pages(d, v_pool, &tv)) return PA_ERR_CUDA;
  DecodeArgs a;
  fill_decode_args(&a, d, plan.split, q, block_tables, context_lens, out, workspace, err_flag,
                   (long long)sms * (d->block_size == 16 ? 2 : 3));
  uint8_t *ws = static_cast<uint8_t *>(workspace) + plan.split.total();
  a.stats = reinterpret_cast<float2 *>(ws);
  a.logits = reinterpret_cast<float *>(ws + plan.stats);
  // One launch where every (sequence, kv head) is a CTA or a cluster, rows are
  // not shared and a CTA's logits are at most 64 KB; else a second kernel, on
  // the whole GPU, adds the weights.  (us in a graph, one launch and two, 8 heads a
  // kv head: four short sequences 4.3 and 5.5; 64 x 1024 tokens, 32 KB a CTA, 50.8
  // and 52.3; 64 x 2048, 64 KB, 91.9 and 93.6; 64 x 4096, 128 KB, 185.0 and 185.7;
  // 64 x 8192 with 4 heads, 128 KB, 344.6 and 341.8; 40 x 8192, 256 KB, 311 and 298;
  // 8 x 32768, 256 KB, 189 and 184: they meet near 128 KB, within 1 % there.)
  const int64_t cta_bytes = (int64_t)plan.split.part_pages * d->block_size * a.G * (int64_t)sizeof(float);
  const bool one = !weight_rows && plan.split.max_parts <= kClusterParts && cta_bytes <= 64 * 1024;
  a.w_in = weights;
  a.w_out = one ? weights_out : nullptr;
  a.max_tokens = (size_t)max_tokens;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // The second kernel reads what the first left in the workspace: no other such
  // call may come between the two on the stream, whatever thread makes it.
  static std::mutex both;
  const std::lock_guard<std::mutex> lock(both);
  const int st = d->head_dim == 128 ? (d->block_size == 16 ? dispatch_logits<128, 16>(d, tk, tv, a, sms, s)
                                                           : dispatch_logits<128, 32>(d, tk, tv, a, sms, s))
                                    : (d->block_size == 16 ? dispatch_logits<64, 16>(d, tk, tv, a, sms, s)
                                                           : dispatch_logits<64, 32>(d, tk, tv, a, sms, s));
  if (st != PA_OK) return st;
  if (one || d->max_context_len == 0) return PA_OK;
  WeightArgs w{};
  w.logits = a.logits;
  w.stats = a.stats;
  w.ctx = context_lens;
  w.rows = weight_rows;
  w.w_in = weights;
  w.w_out = weights_out;
  w.err = err_flag;
  w.S = d->num_seqs;
  w.Hkv = d->num_kv_heads;
  w.G = a.G;
  w.num_rows = num_rows;
  w.max_ctx = d->max_context_len;
  w.max_tokens_table = d->max_blocks_per_seq * d->block_size;
  w.max_tokens = (size_t)max_tokens;
  const int chunks = (d->max_context_len + kWTokens - 1) / kWTokens;
  const size_t smem = weight_rows ? ((size_t)d->num_seqs + kWThreads - 1) / kWThreads * (kWThreads / 8) : 0;
  const dim3 wgrid(chunks, d->num_kv_heads, d->num_seqs);
  auto kern = a.G % 4 == 0 ? weights_kernel<4> : a.G % 2 == 0 ? weights_kernel<2> : weights_kernel<1>;
  return launch_dependent(kern, wgrid, kWThreads, smem, 1, s, w);
}
