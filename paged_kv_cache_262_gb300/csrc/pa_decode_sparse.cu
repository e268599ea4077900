// Block-sparse paged decode attention for sm_103a: every (sequence, kv head)
// attends the keys of the blocks on its own list,
//   out = sum_{j in listed blocks, j < ctx} softmax_j(scale * q.k_j) v_j,
// the attention behind a selection of blocks (pa_block_select.cu).  It serves
// the decode phase of "Configuring vLLM and PagedAttention for High Throughput
// Enterprise LLM Serving" ("Memory Bottlenecks in Autoregressive LLM
// Inference": decode reads the whole cache for every token), whose bytes a
// list of blocks bounds.
//
// The unit is the decode kernel's (pa_decode_body.cuh): the list's blocks are
// resolved through the block table once and streamed by TMA into per-warp
// rings, warp MMAs, online softmax in fp32, the probabilities in two bf16 terms.
// A list has the same length for every sequence, so the split plan is that of
// contexts of num_select blocks and no unit is longer than another; the parts of
// a unit are a cluster and join through shared memory (through the workspace:
// 22 us for the second case below).
//
// The bytes bind: 240 sequences, 24 blocks of 32 tokens each at most, 8 kv heads
// of 128: 107 us, 6.5 TB/s (103 with the probabilities rounded once: with one
// slot a warp the second product is not hidden).  128 blocks of 16 for 8
// sequences, 67 MB: 17.1 us, 3.9 TB/s (16.3 in a graph) -- one wave of 256 CTAs, of which starting,
// three dependent loads, the first gathers and the join are 7 us; more slots a
// warp or other parts (16, 22, 43, 64 pages) are no faster.  One sequence, 256
// blocks, 32 query and 8 kv heads: 10.3 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pa_decode_body.cuh"
#include "pa_internal.h"
#include "pagedattn.h"

namespace pa {
namespace {

template <int D, int B, int NT, int NST, bool CL>
__global__ void __launch_bounds__(128)
    sparse_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const DecodeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  grid_wait();
  grid_launch_dependents();
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int lin = (blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
  decode_unit<D, B, NT, 4, NST, false, false, false, D == 128, true, false, CL>(&tmK, &tmV, a, lin, threadIdx.x, smem,
                                                                                0);
}

template <int D, int B, int NT>
int launch_sparse(const pa_decode_desc *d, const CUtensorMap &tk, const CUtensorMap &tv, const DecodeArgs &a,
                  cudaStream_t st) {
  constexpr int NST = B == 16 ? 2 : 1;
  return launch_parts(sparse_kernel<D, B, NT, NST, false>, sparse_kernel<D, B, NT, NST, true>,
                      DecodeSmem<D, B, 4, NST>::kAlloc, d, 128, tk, tv, a, st);
}

// The desc whose split plan a list of num_select blocks takes.
pa_decode_desc list_desc(const pa_decode_desc *d, int num_select) {
  pa_decode_desc l = *d;
  l.max_context_len = num_select * d->block_size;
  return l;
}

int validate_sparse(const pa_decode_desc *d, int num_select) {
  const int st = validate_decode_desc(d);
  if (st != PA_OK) return st;
  if (num_select <= 0) return PA_ERR_INVALID;
  if (num_select > kMaxParts * kMaxPartPages) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

}  // namespace
}  // namespace pa

extern "C" size_t pa_decode_sparse_workspace_bytes(const pa_decode_desc *d, int num_select) {
  using namespace pa;
  if (validate_sparse(d, num_select) != PA_OK) return 0;
  const pa_decode_desc l = list_desc(d, num_select);
  return make_cluster_plan(&l, current_sm_count()).total();
}

extern "C" int pa_paged_attention_decode_sparse(const pa_decode_desc *d, const void *q, const void *k_pool,
                                                const void *v_pool, const int32_t *block_tables,
                                                const int32_t *context_lens, const int32_t *selected, int num_select,
                                                void *out, void *workspace, size_t workspace_bytes, int32_t *err_flag,
                                                void *stream) {
  using namespace pa;
  const int vs = validate_sparse(d, num_select);
  if (vs != PA_OK) return vs;
  if (d->num_seqs == 0) return PA_OK;
  if (!q || !k_pool || !v_pool || !block_tables || !context_lens || !selected || !out) return PA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out)) return PA_ERR_INVALID;
  if (d->num_seqs > 65535 || d->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  const int sms = current_sm_count();
  if (sms <= 0) return PA_ERR_CUDA;
  const pa_decode_desc l = list_desc(d, num_select);
  const DecodePlan plan = make_cluster_plan(&l, sms);
  if (plan.total() > 0 && (!workspace || workspace_bytes < plan.total() || !aligned16(workspace)))
    return PA_ERR_WORKSPACE;
  CUtensorMap tk, tv;
  if (!encode_kv_pages(d, k_pool, &tk) || !encode_kv_pages(d, v_pool, &tv)) return PA_ERR_CUDA;
  DecodeArgs a;
  fill_decode_args(&a, d, plan, q, block_tables, context_lens, out, workspace, err_flag, 0);
  a.lpt = 0;  // every list has the same length
  a.sel = selected;
  a.nsel = num_select;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool wide = a.G > 8;
  if (d->head_dim == 128) {
    if (d->block_size == 16)
      return wide ? launch_sparse<128, 16, 2>(d, tk, tv, a, s) : launch_sparse<128, 16, 1>(d, tk, tv, a, s);
    return wide ? launch_sparse<128, 32, 2>(d, tk, tv, a, s) : launch_sparse<128, 32, 1>(d, tk, tv, a, s);
  }
  if (d->block_size == 16)
    return wide ? launch_sparse<64, 16, 2>(d, tk, tv, a, s) : launch_sparse<64, 16, 1>(d, tk, tv, a, s);
  return wide ? launch_sparse<64, 32, 2>(d, tk, tv, a, s) : launch_sparse<64, 32, 1>(d, tk, tv, a, s);
}
