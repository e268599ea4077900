// Block selection for sparse decode attention, sm_103a: per-block bounds of
// the cached keys, and the choice of the blocks each (sequence, kv head)
// attends by a cheap score of them.
//
//   lo[b][h][d] = min_j k_j[d],  hi[b][h][d] = max_j k_j[d]   over the block's keys
//   score(s, h, i) = max_g sum_d (q_gd > 0 ? q_gd hi_id : q_gd lo_id)  >=  max_{j in i} q_g.k_j
//
// over the G query heads g of kv head h: no key of a block can have a larger
// product with the query than the block's score.  The score reads 4 D bytes a
// (block, kv head) where attention reads 4 D B, so choosing costs 1/B of what
// attending everything would (decode re-reads the whole cache for each token:
// "Configuring vLLM and PagedAttention for High Throughput Enterprise LLM
// Serving", "Memory Bottlenecks in Autoregressive LLM Inference").
//
// Both read more than they compute.  Bounds of 8 x 32768 tokens (8 kv heads, D
// 128): 92.5 us, 6.5 TB/s; of one step of 64 sequences 2.8 us, a launch.
// Selection of 128 of 2048 blocks for 8 sequences and 64 query heads: 22 us for
// 67 MB, about 12 reading (5.8 TB/s) and 5 selecting, which one CTA a row does
// after the rest; 32 of up to 128 blocks for 64 sequences 9.4 us and 33 of 256
// for one sequence 6.5 us in a graph (6.8-7.5 a call from Python, the host's), in
// which the steps of the selection bind.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_decode_body.cuh"
#include "pa_internal.h"
#include "pa_select.cuh"
#include "pagedattn.h"

namespace pa {
namespace {

// ------------------------------------------------------------- key bounds
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}

struct BoundsArgs {
  const uint4 *k;
  uint4 *bounds;  // [num_blocks][Hkv][2][D]
  const int32_t *bt, *ctx, *start;
  int32_t *err;
  int Hkv, num_blocks, max_blocks, max_ctx, max_new;
};

// grid (8 (block, kv head) runs, sequence); a warp reduces one run.  A run is
// contiguous: every load instruction of the warp covers 512 consecutive bytes.
template <int D, int B>
__global__ void __launch_bounds__(256) key_bounds_kernel(const BoundsArgs a) {
  constexpr int C = D / 8;          // 16-byte chunks of a key
  constexpr int R = 32 / C;         // keys a load instruction covers
  grid_wait();
  grid_launch_dependents();
  const int s = blockIdx.y, lane = threadIdx.x & 31;
  const int unit = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int ctx = __ldg(a.ctx + s), start = a.start ? __ldg(a.start + s) : 0;
  if (ctx <= 0 || ctx > a.max_blocks * B || ctx > a.max_ctx || start < 0 || start > ctx || ctx - start > a.max_new) {
    if (unit == 0 && lane == 0 && a.err) atomicOr(a.err, PA_DEVERR_CTX);
    return;
  }
  const int i = start / B + unit / a.Hkv, h = unit % a.Hkv;
  if (i >= (ctx + B - 1) / B) return;
  const int pg = __ldg(a.bt + (size_t)s * a.max_blocks + i);
  if (pg < 0 || pg >= a.num_blocks) {
    if (lane == 0 && a.err) atomicOr(a.err, PA_DEVERR_PAGE);
    return;
  }
  const size_t run = (size_t)pg * a.Hkv + h;
  const uint4 *k = a.k + run * B * C;
  const int rows = min(B, ctx - i * B);
  uint4 x[B / R];
#pragma unroll
  for (int r = 0; r < B / R; ++r)  // a row past the context: the block's first key once more
    x[r] = __ldcs(k + (r * R + lane / C < rows ? r * 32 + lane : lane % C));
  uint4 lo = x[0], hi = x[0];
#pragma unroll
  for (int r = 1; r < B / R; ++r) {
    lo = make_uint4(min2(lo.x, x[r].x), min2(lo.y, x[r].y), min2(lo.z, x[r].z), min2(lo.w, x[r].w));
    hi = make_uint4(max2(hi.x, x[r].x), max2(hi.y, x[r].y), max2(hi.z, x[r].z), max2(hi.w, x[r].w));
  }
#pragma unroll
  for (int o = C; o < 32; o <<= 1) {
    lo.x = min2(lo.x, __shfl_xor_sync(0xffffffffu, lo.x, o));
    lo.y = min2(lo.y, __shfl_xor_sync(0xffffffffu, lo.y, o));
    lo.z = min2(lo.z, __shfl_xor_sync(0xffffffffu, lo.z, o));
    lo.w = min2(lo.w, __shfl_xor_sync(0xffffffffu, lo.w, o));
    hi.x = max2(hi.x, __shfl_xor_sync(0xffffffffu, hi.x, o));
    hi.y = max2(hi.y, __shfl_xor_sync(0xffffffffu, hi.y, o));
    hi.z = max2(hi.z, __shfl_xor_sync(0xffffffffu, hi.z, o));
    hi.w = max2(hi.w, __shfl_xor_sync(0xffffffffu, hi.w, o));
  }
  if (lane < 2 * C) a.bounds[run * 2 * C + lane] = lane < C ? lo : hi;
}

// -------------------------------------------------------------- selection
constexpr int kSelKeys = 8192;   // keys held in shared memory; more are re-read from the workspace
constexpr int kSelRefine = 128;  // blocks near the threshold that are ranked in shared memory

struct SelectArgs {
  const __nv_bfloat16 *q;
  const uint4 *bounds;
  const int32_t *bt, *ctx;
  int32_t *selected;           // [S][Hkv][k]
  unsigned long long *keys64;  // [S][Hkv][stride]: exact scores (many ties only)
  uint32_t *keys;              // [S][Hkv][stride]: scores as ordered keys (LONG launches only)
  float *span;                 // [S][Hkv][max_chunks]: largest absolute sum of a chunk (LONG launches only)
  unsigned long long *cnt;     // [S][Hkv] arrivals (LONG launches only)
  int32_t *err;
  int Hq, Hkv, G, num_blocks, max_blocks, max_ctx, k, sink, recent, B, max_chunks;
  int chunk;                   // blocks a CTA scores, a multiple of 16 blocks a warp
  size_t stride;
  unsigned int epoch;
};

template <int SW>
struct RowSelect {
  SelectSmem<SW * 32> sm;
  uint4 keys[kSelKeys / 4];
  unsigned long long ex[kSelRefine];
  int exi[kSelRefine];
  float span[8];              // a CTA of the cluster each:
  uint32_t least[8], most[8];  // its least and largest key
  float mx[SW];
  uint32_t wl[SW], wm[SW];
  int nex, last;
};

// A block's score in 64 bits as an ordered key, by one warp: every product of
// two bf16 values is exact, and blocks of equal bounds get equal sums.  The
// heads whose fp32 sum is more than `slack` below the largest cannot be the
// maximum (slack covers twice the error of a plain fp32 sum; infinite: every
// head is summed in 64 bits).
template <int D, int H>  // H: heads, at least G
__device__ unsigned long long exact_score(const SelectArgs &a, const __nv_bfloat16 *q, int pg, int h, float slack,
                                          int lane) {
  constexpr int P = D / 32;  // elements of a lane, a multiple of two
  const __nv_bfloat16 *lo = reinterpret_cast<const __nv_bfloat16 *>(a.bounds) + ((size_t)pg * a.Hkv + h) * 2 * D;
  float bl[P], bh[P];
#pragma unroll
  for (int p = 0; p < P; p += 2) {
    const uint32_t l = __ldg(reinterpret_cast<const uint32_t *>(lo + lane * P + p));
    const uint32_t u = __ldg(reinterpret_cast<const uint32_t *>(lo + D + lane * P + p));
    bl[p] = bf16_lo(l), bl[p + 1] = bf16_hi(l);
    bh[p] = bf16_lo(u), bh[p + 1] = bf16_hi(u);
  }
  float fs[H], top = -INFINITY;
  uint32_t qv[H][P / 2];
#pragma unroll
  for (int g = 0; g < H; ++g) {
    fs[g] = 0.f;
#pragma unroll
    for (int p = 0; p < P; p += 2)
      qv[g][p / 2] = g < a.G ? __ldg(reinterpret_cast<const uint32_t *>(q + g * D + lane * P + p)) : 0u;
  }
#pragma unroll
  for (int g = 0; g < H; ++g)
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const float x = p & 1 ? bf16_hi(qv[g][p / 2]) : bf16_lo(qv[g][p / 2]);
      fs[g] += x * (x > 0.f ? bh[p] : bl[p]);
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int g = 0; g < H; ++g) fs[g] += __shfl_xor_sync(0xffffffffu, fs[g], o);
#pragma unroll
  for (int g = 0; g < H; ++g)
    if (g < a.G) top = fmaxf(top, fs[g]);
  unsigned long long best = 0ull;
#pragma unroll
  for (int g = 0; g < H; ++g) {
    if (g >= a.G || fs[g] < top - slack) continue;  // (the same for every lane)
    double sum = 0.0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const float x = p & 1 ? bf16_hi(qv[g][p / 2]) : bf16_lo(qv[g][p / 2]);
      if (x != 0.f) sum += (double)x * (double)(x > 0.f ? bh[p] : bl[p]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const unsigned long long k = order_key64(sum);
    best = k > best ? k : best;
  }
  return best;
}

// How far an fp32 score may be from the exact one, as a part of the largest
// absolute sum A = sum_d |q_gd b_d| of the row: each of the 2 D / 16 MMAs adds
// 17 terms no larger than A, each, and the sum, cut at 2^-23 of the largest of
// them or better (and A itself, of the same MMAs, may be short by as much of itself).
template <int D>
constexpr float kScoreError = 18.f * (2 * D / 16) * 1.1920929e-07f * 1.001f;

// One CTA selects a row's blocks from its keys (in r.keys, or past kSelKeys of
// them in the workspace), A the row's largest absolute sum; least and most: the
// least and largest key of some of them, all among the threads.
template <int D, int NT, int SW, bool LONG>
__device__ void select_row(const SelectArgs &a, RowSelect<SW> &r, size_t row, int s, int h, int n, float A,
                           uint32_t least, uint32_t most, int tid) {
  constexpr int kThreads = SW * 32;
  const int lane = tid & 31, warp = tid >> 5;
  const int first = a.sink, end = n - a.recent;
  const int32_t *bt = a.bt + (size_t)s * a.max_blocks;
  const __nv_bfloat16 *q = a.q + ((size_t)s * a.Hq + (size_t)h * a.G) * D;
  int32_t *out = a.selected + row * a.k;
  const int N = end - first, want = a.k - a.sink - a.recent;
  for (int i = tid; i < a.sink; i += kThreads) out[i] = i;
  for (int i = tid; i < a.recent; i += kThreads) out[a.k - a.recent + i] = end + i;
  if (want == 0) return;
  const bool in_smem = !LONG || N <= kSelKeys;
  uint32_t *keys = in_smem ? reinterpret_cast<uint32_t *>(r.keys) : a.keys + row * a.stride;
  auto key4 = [&](int i) { return keys4(in_smem ? r.keys[i / 4] : __ldcg(reinterpret_cast<const uint4 *>(keys + i))); };
  auto key1 = [&](int i) {
    return in_smem ? reinterpret_cast<const uint32_t *>(r.keys)[i] : __ldcg(keys + i);
  };
  const float slack = 2.f * kScoreError<D> * A + 1e-30f;  // (and what products below fp32's normal range lose)
  const bool finite = slack < INFINITY;  // false for NaN too: then no fp32 score is trusted
  uint32_t lo = 0u, hi = 0xfffffffeu;    // (no score's key is above it)
  int above = 0;
  if (finite) {
    const Kth<uint32_t> t = N <= kThreads ? kth_of_few<kThreads, uint32_t>(key4, key1, N, want, r.sm, tid)
                                          : kth_largest<kThreads, uint32_t>(key4, N, want, r.sm, tid, least, most);
    above = t.above;
    if (t.key != 0u) {
      const float v = key_value(t.key);
      lo = order_key(__fsub_rd(v, slack));
      hi = order_key(__fadd_ru(v, slack));
    } else {
      hi = 0u;  // blocks outside the pool are among the chosen: those that can be read all are
    }
  }
  auto emit = [&](int pos, int i, uint32_t) { out[a.sink + pos] = first + i; };
  if (hi == 0u) {  // (of blocks outside the pool, the first)
    take_above<kThreads, uint32_t>(key4, key1, N, 0u, want - above, want, r.sm, tid, emit);
    return;
  }
  // blocks above hi are chosen whatever their rounding, those below lo are not:
  // a count of either kind for each warp's stretch, and a list of those between
  const Stretch<kThreads> w(N, warp);
  int gt = 0, nr = 0;
#pragma unroll 2
  for (int i = w.beg + 4 * lane; i < w.end; i += 128) {
    const Keys4<uint32_t> k = key4(i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (i + e >= w.end || k.v[e] < lo) continue;
      if (k.v[e] > hi) {
        ++gt;
      } else {
        ++nr;
        const int at = atomicAdd(&r.nex, 1);
        if (at < kSelRefine) r.exi[at] = i + e;
      }
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  nr = __reduce_add_sync(0xffffffffu, nr);
  if (lane == 0) {
    r.sm.a[warp] = gt;
    r.sm.b[warp] = nr;
  }
  __syncthreads();
  const int near_ = r.nex, need = want - sum_all<kThreads>(r.sm.a, lane);
  int pos = sum_before<kThreads>(r.sm.a, lane, warp);
  if (near_ == need) {
    pos += sum_before<kThreads>(r.sm.b, lane, warp);
    list_stretch<kThreads, uint32_t>(key1, w, lo, true, 0, 0, pos, want, lane, emit);
    return;
  }
  if (near_ <= kSelRefine) {  // few: their exact scores, ranked by counting
    for (int c = warp; c < near_; c += SW) {
      const int pg = __ldg(bt + first + r.exi[c]);
      const bool ok = pg >= 0 && pg < a.num_blocks;
      const unsigned long long x = ok ? exact_score<D, 8 * NT>(a, q, pg, h, slack, lane) : 0ull;
      if (lane == 0) r.ex[c] = x;
    }
    __syncthreads();
    static_assert(kSelRefine <= kThreads, "a thread a block");
    int rank = 0;
    if (tid < near_) {
      const unsigned long long x = r.ex[tid];
      const int xi = r.exi[tid];
      for (int o = 0; o < near_; ++o) rank += r.ex[o] > x || (r.ex[o] == x && r.exi[o] < xi);
      keys[xi] = rank < need ? 0xffffffffu : 0u;
    }
    __syncthreads();
    if (tid < near_ && rank >= need) r.exi[tid] = N;  // not one of the chosen
    __syncthreads();
    int before = 0;  // chosen ones in the stretches before this warp's
    for (int c = lane; c < near_; c += 32) before += r.exi[c] < w.beg;
    pos += __reduce_add_sync(0xffffffffu, before);
    list_stretch<kThreads, uint32_t>(key1, w, hi + 1u, true, 0, 0, pos, want, lane, emit);
    return;
  }
  // many (scores that tie in numbers, infinite bounds): 64-bit keys for all of
  // them in the workspace
  unsigned long long *k64 = a.keys64 + row * a.stride;
  for (int i = warp; i < N; i += SW) {
    const uint32_t k = key1(i);
    unsigned long long x = k > hi ? ~0ull : 0ull;
    if (k >= lo && k <= hi) {
      const int pg = __ldg(bt + first + i);
      const bool ok = pg >= 0 && pg < a.num_blocks;
      x = ok ? exact_score<D, 8 * NT>(a, q, pg, h, slack, lane) : 1ull;
    }
    if (lane == 0) k64[i] = x;
  }
  __threadfence_block();
  __syncthreads();
  auto key64 = [&](int i) {
    Keys4<unsigned long long> k;
#pragma unroll
    for (int e = 0; e < 4; ++e) k.v[e] = i + e < N ? k64[i + e] : 0ull;
    return k;
  };
  unsigned long long l64 = ~0ull, m64 = 0ull;
  for_keys<kThreads, unsigned long long>(key64, N, tid, [&](int, unsigned long long k) {
    l64 = min(l64, k);
    m64 = max(m64, k);
  });
  const Kth<unsigned long long> t = kth_largest<kThreads, unsigned long long>(key64, N, want, r.sm, tid, l64, m64);
  take_above<kThreads, unsigned long long>(key64, [&](int i) { return k64[i]; }, N, t.key, want - t.above, want, r.sm, tid,
                                           [&](int pos, int i, unsigned long long) { out[a.sink + pos] = first + i; });
}

// grid (chunk, kv head, sequence).  Every CTA scores its chunk of a row.  The
// chunks of a row are a cluster: the scores go straight into the shared memory
// of its first CTA, which selects (by way of the workspace, an arrival counter
// and the last CTA to arrive this handing over took 4.6 us, not 0.7).  LONG: rows of
// more blocks than that holds, by way of the workspace.
template <int D, int NT, int SW, bool LONG>
__global__ void __launch_bounds__(SW * 32, (NT == 1 ? 16 : 8) / SW) select_kernel(const SelectArgs a) {
  constexpr int CH = 2 * D / 32;  // 32-element steps over a block's bounds (lo, then hi)
  constexpr int kThreads = SW * 32;
  __shared__ RowSelect<SW> r;
  const int chunk = blockIdx.x, h = blockIdx.y, s = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = a.B;
  const size_t row = (size_t)s * a.Hkv + h;
  grid_wait();
  const int ctx = __ldg(a.ctx + s);
  const bool bad = ctx <= 0 || ctx > a.max_blocks * B || ctx > a.max_ctx;
  const int n = bad ? 0 : (ctx + B - 1) / B;
  // The blocks listed whatever their score, the first `lead` and those from `tail`
  // on, have their entries looked at once a sequence, by its first CTA; those that
  // compete, where they are scored.
  const int32_t *bt = a.bt + (size_t)s * a.max_blocks;
  auto look = [&](int lead, int tail) {
    if (chunk != 0 || h != 0 || !a.err) return;
    for (int i = tid; i < lead + n - tail; i += kThreads) {
      const int pg = __ldg(bt + (i < lead ? i : tail + i - lead));
      if (pg < 0 || pg >= a.num_blocks) atomicOr(a.err, PA_DEVERR_PAGE);
    }
  };
  if (n <= a.k) {  // every block, or none (the same for the whole cluster)
    look(0, 0);
    if (chunk == 0) {
      int32_t *out = a.selected + row * a.k;
      for (int i = tid; i < a.k; i += kThreads) out[i] = i < n ? i : -1;
      if (bad && h == 0 && tid == 0 && a.err) atomicOr(a.err, PA_DEVERR_CTX);
    }
    return;
  }
  const int nchunks = (n + a.chunk - 1) / a.chunk;
  const bool clustered = !LONG && gridDim.x > 1;
  if (LONG && chunk >= nchunks) return;
  // the first CTA's shared memory must be there before another writes to it
  if (clustered) cluster_arrive();
  const int first = a.sink, end = n - a.recent;  // the blocks that compete
  const __nv_bfloat16 *q = a.q + ((size_t)s * a.Hq + (size_t)h * a.G) * D;
  const int i_end = min(end, (chunk + 1) * a.chunk);

  // lane l's block of a tile: row l / 4 and that + 8; -1: outside the pool, -2:
  // not competing
  auto page = [&](int i) -> int { return i >= first && i < i_end ? max(__ldg(bt + i), -1) : -2; };
  int i0 = chunk * a.chunk + warp * 16;
  int pg[2] = {page(i0 + (lane >> 2)), page(i0 + 8 + (lane >> 2))};

  // ---- scores of this CTA's blocks: S[block][head] = [lo hi] . [q- q+], the
  // contraction in whatever order of d suits the loads (lane t of a quad takes
  // the 16-byte chunks t, t + 4, ...), the same for both operands; and the
  // same of the absolute values, by which the score's error is bounded.
  uint32_t qf[NT][CH / 2][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int g = nt * 8 + (lane >> 2);
#pragma unroll
    for (int c = 0; c < CH / 2; ++c) {
      const uint4 v = g < a.G ? __ldg(reinterpret_cast<const uint4 *>(q + (size_t)g * D) + c * 4 + (lane & 3))
                              : make_uint4(0u, 0u, 0u, 0u);
      qf[nt][c][0] = v.x;
      qf[nt][c][1] = v.y;
      qf[nt][c][2] = v.z;
      qf[nt][c][3] = v.w;
    }
  }
  if (tid == 0) r.nex = 0;
  if (clustered) cluster_wait();
  uint32_t *keys = LONG ? a.keys + row * a.stride : reinterpret_cast<uint32_t *>(r.keys);
  const uint32_t keys0 = clustered ? cluster_addr(smem_u32(r.keys), 0) : smem_u32(r.keys);
  float span = 0.f;
  uint32_t least = ~0u, most = 0u;
  for (; i0 < i_end; i0 += 16 * SW) {
    uint4 x[2][CH];
    bool have[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      have[e] = pg[e] >= 0 && pg[e] < a.num_blocks;
      if (!have[e] && pg[e] != -2 && a.err) atomicOr(a.err, PA_DEVERR_PAGE);
      const uint4 *src = a.bounds + ((size_t)(have[e] ? pg[e] : 0) * a.Hkv + h) * (D / 4) + (lane & 3);
#pragma unroll
      for (int c = 0; c < CH; ++c) x[e][c] = have[e] ? __ldg(src + 4 * c) : make_uint4(0u, 0u, 0u, 0u);
    }
    const int next = i0 + 16 * SW + (lane >> 2);
    pg[0] = page(next);
    pg[1] = page(next + 8);
    float acc[NT][4], abs_[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
      abs_[nt][0] = abs_[nt][1] = abs_[nt][2] = abs_[nt][3] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint4 u = x[0][c], v = x[1][c];
      const uint32_t a0[4] = {u.x, v.x, u.y, v.y}, a1[4] = {u.z, v.z, u.w, v.w};
      uint32_t p0[4], p1[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) p0[e] = a0[e] & 0x7fff7fffu, p1[e] = a1[e] & 0x7fff7fffu;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          b[e] = c < CH / 2 ? min2(qf[nt][c % (CH / 2)][e], 0u) : max2(qf[nt][c % (CH / 2)][e], 0u);
        mma_16816(acc[nt], a0, b[0], b[1]);
        mma_16816(acc[nt], a1, b[2], b[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] &= 0x7fff7fffu;
        mma_16816(abs_[nt], p0, b[0], b[1]);
        mma_16816(abs_[nt], p1, b[2], b[3]);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float best = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int g = nt * 8 + 2 * (lane & 3);
        if (g < a.G) best = fmaxf(best, acc[nt][2 * e]);
        if (g + 1 < a.G) best = fmaxf(best, acc[nt][2 * e + 1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // (heads past G: 0)
          const float y = abs_[nt][2 * e + k];
          span = y <= 3.4028235e38f ? fmaxf(span, y) : INFINITY;
        }
      }
      best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1));
      best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 2));
      const int i = i0 + (lane >> 2) + 8 * e;
      if ((lane & 3) == 0 && i >= first && i < i_end) {
        const uint32_t k = have[e] ? order_key(best) : 0u;
        least = min(least, k);
        most = max(most, k);
        if (LONG)
          keys[i - first] = k;
        else if (clustered)
          cluster_store(keys0 + 4 * (i - first), k);
        else
          keys[i - first] = k;
      }
    }
  }
  look(first, end);  // (here the scores have left the table in L1: 0.1 us less than before them)
  grid_launch_dependents();
  const bool one = !LONG && !clustered;  // then the threads' own least and largest keys will do
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) span = fmaxf(span, __shfl_xor_sync(0xffffffffu, span, o));
  if (lane == 0) r.mx[warp] = span;
  if (!LONG && !one) {
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) r.wl[warp] = least, r.wm[warp] = most;
  }
  if (LONG) __threadfence();
  __syncthreads();
#pragma unroll
  for (int w = 0; w < SW; ++w) span = fmaxf(span, r.mx[w]);
  if (!LONG) {
    if (clustered) {
      if (tid == 0) {
#pragma unroll
        for (int w = 0; w < SW; ++w) least = min(least, r.wl[w]), most = max(most, r.wm[w]);
        cluster_store(cluster_addr(smem_u32(&r.span[chunk]), 0), __float_as_uint(span));
        cluster_store(cluster_addr(smem_u32(&r.least[chunk]), 0), least);
        cluster_store(cluster_addr(smem_u32(&r.most[chunk]), 0), most);
      }
      cluster_arrive();
      if (chunk != 0) return;
      cluster_wait();
      for (int c = 0; c < (int)gridDim.x; ++c) {
        span = fmaxf(span, r.span[c]);
        least = min(least, r.least[c]);
        most = max(most, r.most[c]);
      }
    }
    select_row<D, NT, SW, LONG>(a, r, row, s, h, n, span, least, most, tid);
    return;
  }
  if (tid == 0) {
    a.span[row * a.max_chunks + chunk] = span;
    __threadfence();
    r.last = arrive_count(a.cnt + row, a.epoch) == (unsigned int)nchunks;
  }
  __syncthreads();
  if (!r.last) return;
  __threadfence();
  if (tid == 0) a.cnt[row] = 0ull;
  const int N = end - first;
  if (N <= kSelKeys) {
    const uint4 *src = reinterpret_cast<const uint4 *>(a.keys + row * a.stride);
    for (int i = tid; i < (N + 3) / 4; i += kThreads) r.keys[i] = __ldcg(src + i);
  }
  for (int c = lane; c < nchunks; c += 32) span = fmaxf(span, __ldcg(a.span + row * a.max_chunks + c));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) span = fmaxf(span, __shfl_xor_sync(0xffffffffu, span, o));
  least = ~0u, most = 0u;
  for (int i = tid; i < N; i += kThreads) {
    const uint32_t k = __ldcg(a.keys + row * a.stride + i);
    least = min(least, k);
    most = max(most, k);
  }
  __syncthreads();
  select_row<D, NT, SW, LONG>(a, r, row, s, h, n, span, least, most, tid);
}

// Rows of at most kSelKeys blocks: a cluster of 1, 2, 4 or 8 CTAs a row, as
// many as make about two CTAs an SM and leave every warp a tile; CTAs of four
// warps where the rows alone are more than two an SM.  Longer rows: chunks of
// 128 blocks and more.
struct SelectPlan {
  bool rows_long = false;
  int warps = 8, chunk = 0, max_chunks = 0;
  size_t stride = 0, keys = 0, keys64 = 0, span = 0, cnt = 0;
  size_t total() const { return keys + keys64 + span + cnt; }
};

SelectPlan make_select_plan(const pa_decode_desc *d, int sms) {
  SelectPlan p;
  const int64_t B = d->block_size;
  const size_t nblk = (size_t)std::max<int64_t>(1, ((int64_t)d->max_context_len + B - 1) / B);
  const size_t rows = (size_t)d->num_seqs * d->num_kv_heads, slots = 2 * (size_t)std::max(sms, 1);
  auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
  p.rows_long = nblk > kSelKeys;
  p.warps = !p.rows_long && rows > slots ? 4 : 8;
  const size_t unit = 16 * p.warps;
  if (p.rows_long) {  // as many CTAs as fill the slots once, each of up to 8 tiles a warp
    const size_t per = (rows * nblk + slots - 1) / slots;
    p.chunk = (int)std::min<size_t>(8 * unit, std::max<size_t>(1, (per + unit - 1) / unit) * unit);
    p.max_chunks = (int)((nblk + p.chunk - 1) / p.chunk);
  } else {
    size_t c = 1;
    while (c < 8 && rows * c * 2 <= slots && c * unit < nblk) c *= 2;
    p.chunk = (int)(((nblk + c - 1) / c + unit - 1) / unit * unit);
    p.max_chunks = (int)c;
  }
  p.stride = (nblk + 3) & ~(size_t)3;
  p.keys64 = up(rows * p.stride * 8);
  if (p.rows_long) {
    p.keys = up(rows * p.stride * 4);
    p.span = up(rows * ((nblk + unit - 1) / unit) * 4);  // (whatever the SM count)
    p.cnt = up(rows * 8);
  }
  return p;
}

template <int D, int NT, int SW, bool LONG>
int launch_select(const SelectArgs &a, dim3 grid, cudaStream_t st) {
  auto kern = select_kernel<D, NT, SW, LONG>;
  static_assert(sizeof(RowSelect<SW>) <= 48 * 1024, "static shared memory");
  return launch_dependent(kern, grid, SW * 32, 0, LONG ? 1 : (int)grid.x, st, a);
}

template <int D, int NT>
int dispatch_select(const SelectArgs &a, const SelectPlan &p, dim3 grid, cudaStream_t st) {
  if (p.rows_long) return launch_select<D, NT, 8, true>(a, grid, st);
  return p.warps == 4 ? launch_select<D, NT, 4, false>(a, grid, st) : launch_select<D, NT, 8, false>(a, grid, st);
}

}  // namespace
}  // namespace pa

extern "C" int pa_block_key_bounds(const pa_decode_desc *d, const void *k_pool, const int32_t *block_tables,
                                   const int32_t *context_lens, const int32_t *start_lens, int max_new_tokens,
                                   void *bounds, int32_t *err_flag, void *stream) {
  using namespace pa;
  const int vs = validate_decode_desc(d);
  if (vs != PA_OK) return vs;
  if (max_new_tokens < 0) return PA_ERR_INVALID;
  if (d->num_seqs == 0) return PA_OK;
  if (!k_pool || !block_tables || !context_lens || !bounds || !aligned16(k_pool) || !aligned16(bounds))
    return PA_ERR_INVALID;
  if (d->num_seqs > 65535) return PA_ERR_UNSUPPORTED;
  BoundsArgs a{};
  a.k = static_cast<const uint4 *>(k_pool);
  a.bounds = static_cast<uint4 *>(bounds);
  a.bt = block_tables;
  a.ctx = context_lens;
  a.start = start_lens;
  a.err = err_flag;
  a.Hkv = d->num_kv_heads;
  a.num_blocks = d->num_blocks;
  a.max_blocks = d->max_blocks_per_seq;
  a.max_ctx = d->max_context_len;
  a.max_new = max_new_tokens;
  // most blocks that max_new tokens at the end of a context touch
  const int64_t B = d->block_size;
  const int64_t most = std::max<int64_t>(
      1, std::min<int64_t>((std::min<int64_t>(max_new_tokens, d->max_context_len) + B - 1) / B + 1,
                           ((int64_t)d->max_context_len + B - 1) / B));
  const int64_t gx = (most * d->num_kv_heads + 7) / 8;
  if (gx > 0x7fffffff) return PA_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)gx, d->num_seqs);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto kern = d->head_dim == 128 ? (d->block_size == 16 ? key_bounds_kernel<128, 16> : key_bounds_kernel<128, 32>)
                                 : (d->block_size == 16 ? key_bounds_kernel<64, 16> : key_bounds_kernel<64, 32>);
  return launch_dependent(kern, grid, 256, 0, 1, s, a);
}

extern "C" size_t pa_select_blocks_workspace_bytes(const pa_decode_desc *d) {
  using namespace pa;
  if (validate_decode_desc(d) != PA_OK) return 0;
  return make_select_plan(d, 1).total();
}

extern "C" int pa_select_blocks(const pa_decode_desc *d, const void *q, const void *bounds,
                                const int32_t *block_tables, const int32_t *context_lens, int num_select,
                                int sink_blocks, int recent_blocks, int32_t *selected, void *workspace,
                                size_t workspace_bytes, int32_t *err_flag, void *stream) {
  using namespace pa;
  const int vs = validate_decode_desc(d);
  if (vs != PA_OK) return vs;
  if (num_select <= 0 || sink_blocks < 0 || recent_blocks < 0 || (int64_t)sink_blocks + recent_blocks > num_select)
    return PA_ERR_INVALID;
  if (d->num_seqs == 0) return PA_OK;
  if (!q || !bounds || !block_tables || !context_lens || !selected || !aligned16(q) || !aligned16(bounds))
    return PA_ERR_INVALID;
  if (d->num_seqs > 65535 || d->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < make_select_plan(d, 1).total() || !aligned16(workspace))
    return PA_ERR_WORKSPACE;
  const int sms = current_sm_count();
  if (sms <= 0) return PA_ERR_CUDA;
  const SelectPlan p = make_select_plan(d, sms);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  SelectArgs a{};
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.bounds = static_cast<const uint4 *>(bounds);
  a.bt = block_tables;
  a.ctx = context_lens;
  a.selected = selected;
  a.keys64 = reinterpret_cast<unsigned long long *>(ws);
  a.keys = reinterpret_cast<uint32_t *>(ws + p.keys64);
  a.span = reinterpret_cast<float *>(ws + p.keys64 + p.keys);
  a.cnt = reinterpret_cast<unsigned long long *>(ws + p.keys64 + p.keys + p.span);
  a.err = err_flag;
  a.Hq = d->num_q_heads;
  a.Hkv = d->num_kv_heads;
  a.G = d->num_q_heads / d->num_kv_heads;
  a.num_blocks = d->num_blocks;
  a.max_blocks = d->max_blocks_per_seq;
  a.max_ctx = d->max_context_len;
  a.k = num_select;
  a.sink = sink_blocks;
  a.recent = recent_blocks;
  a.B = d->block_size;
  a.max_chunks = p.max_chunks;
  a.chunk = p.chunk;
  a.stride = p.stride;
  a.epoch = next_decode_epoch();
  const dim3 grid(p.max_chunks, d->num_kv_heads, d->num_seqs);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->head_dim == 128)
    return a.G <= 8 ? dispatch_select<128, 1>(a, p, grid, s) : dispatch_select<128, 2>(a, p, grid, s);
  return a.G <= 8 ? dispatch_select<64, 1>(a, p, grid, s) : dispatch_select<64, 2>(a, p, grid, s);
}
