// Selection of the largest of n keys by one CTA: the threshold by radix
// counting in shared memory, then the taken indices in increasing order.
// Used by the block selection (pa_block_select.cu) and the eviction
// (pa_evict.cu).
#pragma once

#include <stdint.h>

namespace pa {
namespace {

// A 32-bit key that orders as the float does; -0 as +0, NaN above all.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
// The same in 64 bits; NaN as +infinity.
__device__ __forceinline__ unsigned long long order_key64(double x) {
  if (x != x) x = INFINITY;
  const unsigned long long b = (unsigned long long)__double_as_longlong(x + 0.0);
  return (b >> 63) ? ~b : b | (1ull << 63);
}

// Counting bins of a CTA of NT threads: eight a thread.
template <int NT>
constexpr int kDigitBits = NT >= 1024 ? 13 : NT >= 512 ? 12 : 11;
constexpr int kNearKeys = 256;  // keys of one bin that are ranked by comparing all of them

template <int NT>
struct SelectSmem {
  int4 hist[2 * NT];
  unsigned long long lo[NT / 32], hi[NT / 32];
  unsigned long long near_[kNearKeys], kth;
  int a[NT / 32], b[NT / 32];
  int bin, above, count, filled, kth_above;
};

// The want-th largest key (1 <= want <= n) and how many keys are above it.
template <class T>
struct Kth {
  T key;
  int above;
};

__device__ __forceinline__ int lead_zeros(uint32_t x) { return __clz((int)x); }
__device__ __forceinline__ int lead_zeros(unsigned long long x) { return __clzll((long long)x); }

// Whole CTA of NT threads; key(i) for i < n; lo and hi: the least and largest
// key of those that this thread looked at, all of them among the threads.  A
// digit is the bits below those that all keys left share, so that the first
// one already tells keys of one magnitude apart (scores of a context differ in
// few high bits); once a bin's keys are few they are ranked by comparison.
template <int NT, class T, class KeyF>
__device__ Kth<T> kth_largest(KeyF key, int n, int want, SelectSmem<NT> &sm, int tid, T lo, T hi) {
  constexpr int kBits = 8 * sizeof(T), kDigit = kDigitBits<NT>, kBins = 1 << kDigit, kPer = kBins / NT;
  static_assert(kBins * (int)sizeof(int) == (int)sizeof(sm.hist), "eight bins a thread");
  const int lane = tid & 31, warp = tid >> 5;
  int *hist = reinterpret_cast<int *>(sm.hist);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const T l2 = __shfl_xor_sync(0xffffffffu, lo, o), h2 = __shfl_xor_sync(0xffffffffu, hi, o);
    lo = l2 < lo ? l2 : lo;
    hi = h2 > hi ? h2 : hi;
  }
  __syncthreads();  // sm may be in use by a call before
  if (lane == 0) {
    sm.lo[warp] = lo;
    sm.hi[warp] = hi;
  }
  for (int i = tid; i < kBins / 4; i += NT) sm.hist[i] = make_int4(0, 0, 0, 0);
  if (tid == 0) sm.filled = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    lo = (T)sm.lo[w] < lo ? (T)sm.lo[w] : lo;
    hi = (T)sm.hi[w] > hi ? (T)sm.hi[w] : hi;
  }
  int open = kBits - (lo == hi ? kBits : lead_zeros(lo ^ hi));  // low bits in which the keys left differ
  T base = open == kBits ? (T)0 : (hi >> open) << open;
  int left = want, above = 0;
  while (open > 0) {
    const int w = min(kDigit, open), sh = open - w;
#pragma unroll 4
    for (int i = tid; i < n; i += NT) {
      const T k = key(i);
      if (open == kBits || (k ^ base) >> open == 0) atomicAdd(&hist[(int)(k >> sh) & ((1 << w) - 1)], 1);
    }
    __syncthreads();
    // bins from the highest down, kPer consecutive ones a thread
    int cnt[kPer], c = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) c += cnt[j] = hist[kBins - 1 - tid * kPer - j];
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sm.a[warp] = incl;
    __syncthreads();
    int run = incl - c;
    for (int v = 0; v < warp; ++v) run += sm.a[v];
    if (left > run && left <= run + c) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (left > run && left <= run + cnt[j]) {
          sm.bin = kBins - 1 - tid * kPer - j;
          sm.above = run;
          sm.count = cnt[j];
        }
        run += cnt[j];
      }
    }
    for (int i = tid; i < kBins / 4; i += NT) sm.hist[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    base |= (T)sm.bin << sh;
    above += sm.above;
    left -= sm.above;
    open = sh;
    const int count = sm.count;
    if (open > 0 && count <= kNearKeys) {
#pragma unroll 4
      for (int i = tid; i < n; i += NT) {
        const T k = key(i);
        if ((k ^ base) >> open == 0) {
          const int at = atomicAdd(&sm.filled, 1);
          if (at < kNearKeys) sm.near_[at] = k;
        }
      }
      __syncthreads();
      if (tid < count) {
        const T mine = (T)sm.near_[tid];
        int gt = 0, ge = 0;
        for (int j = 0; j < count; ++j) {
          const T o = (T)sm.near_[j];
          gt += o > mine;
          ge += o >= mine;
        }
        if (gt < left && left <= ge) {  // (equal keys write the same)
          sm.kth = mine;
          sm.kth_above = gt;
        }
      }
      __syncthreads();
      return Kth<T>{(T)sm.kth, above + sm.kth_above};
    }
  }
  return Kth<T>{base, above};
}

// Calls emit(position, i) for every i < n with key(i) > t, and for the first
// need of those with key(i) == t, in increasing order of i, at most `room` of
// them (keys that another launch overwrites meanwhile must not write past the
// list).  Whole CTA.
template <int NT, class T, class KeyF, class Emit>
__device__ void take_above(KeyF key, int n, T t, int need, int room, SelectSmem<NT> &sm, int tid, Emit emit) {
  const int lane = tid & 31, warp = tid >> 5;
  const int seg = (n + NT - 1) / NT * 32;  // a warp's consecutive keys
  const int beg = min(n, warp * seg), end = min(n, beg + seg);
  int gt = 0, eq = 0;
  for (int i = beg + lane; i < beg + seg; i += 32) {
    const T k = i < end ? key(i) : (T)0;
    gt += __popc(__ballot_sync(0xffffffffu, i < end && k > t));
    eq += __popc(__ballot_sync(0xffffffffu, i < end && k == t));
  }
  __syncthreads();
  if (lane == 0) {
    sm.a[warp] = gt;
    sm.b[warp] = eq;
  }
  __syncthreads();
  gt = eq = 0;
  for (int w = 0; w < warp; ++w) {
    gt += sm.a[w];
    eq += sm.b[w];
  }
  int pos = gt + min(eq, need);
  const unsigned int below = (1u << lane) - 1u;
  for (int i = beg + lane; i < beg + seg; i += 32) {
    const T k = i < end ? key(i) : (T)0;
    const unsigned int e = __ballot_sync(0xffffffffu, i < end && k == t);
    const bool in = i < end && (k > t || (k == t && eq + __popc(e & below) < need));
    const unsigned int b = __ballot_sync(0xffffffffu, in);
    const int at = pos + __popc(b & below);
    if (in && at < room) emit(at, i);
    pos += __popc(b);
    eq += __popc(e);
  }
}

}  // namespace
}  // namespace pa
