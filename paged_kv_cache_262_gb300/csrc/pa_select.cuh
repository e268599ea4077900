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

// Counting bins of a CTA of NT threads: eight a thread, or sixteen.
template <int NT>
constexpr int kDigitBits = NT >= 1024 ? 13 : NT >= 512 ? 12 : 11;
constexpr int kNearKeys = 256;  // keys of one bin that are ranked by comparing all of them

template <int NT>
struct SelectSmem {
  int4 hist[(1 << kDigitBits<NT>) / 4];
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

// Four consecutive keys: key4(i) for i a multiple of 4 below n (what it gives
// for places past n - 1 is not looked at).
template <class T>
struct Keys4 {
  T v[4];
};

__device__ __forceinline__ Keys4<uint32_t> keys4(uint4 x) { return Keys4<uint32_t>{{x.x, x.y, x.z, x.w}}; }

__device__ __forceinline__ int lead_zeros(uint32_t x) { return __clz((int)x); }
__device__ __forceinline__ int lead_zeros(unsigned long long x) { return __clzll((long long)x); }

// f(i, key) for every key of this thread: four consecutive ones at a time.
template <int NT, class T, class Key4, class F>
__device__ __forceinline__ void for_keys(Key4 key4, int n, int tid, F f) {
#pragma unroll 2
  for (int i = 4 * tid; i < n; i += 4 * NT) {
    const Keys4<T> k = key4(i);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n) f(i + e, k.v[e]);
  }
}

// Whole CTA of NT threads; lo and hi: the least and largest key of those that
// this thread looked at, all of them among the threads.  A digit is the bits
// below those that all keys left share, so that the first one already tells
// keys of one magnitude apart (scores of a context differ in few high bits);
// once a bin's keys are few they are ranked by comparison.
template <int NT, class T, class Key4>
__device__ Kth<T> kth_largest(Key4 key4, int n, int want, SelectSmem<NT> &sm, int tid, T lo, T hi) {
  constexpr int kBits = 8 * sizeof(T), kDigit = kDigitBits<NT>, kBins = 1 << kDigit, kPer = kBins / NT;
  static_assert(kBins * (int)sizeof(int) <= (int)sizeof(sm.hist), "the bins fit");
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
    const bool all = open == kBits;  // (a shift by every bit is none)
    for_keys<NT, T>(key4, n, tid, [&](int, T k) {
      if (all || (k ^ base) >> open == 0) atomicAdd(&hist[(int)(k >> sh) & ((1 << w) - 1)], 1);
    });
    __syncthreads();
    // bins from the highest down, kPer consecutive ones a thread
    int cnt[kPer], c = 0;
#pragma unroll
    for (int j = 0; j < kPer / 4; ++j) {
      const int4 b = sm.hist[(kBins - tid * kPer) / 4 - 1 - j];
      cnt[4 * j] = b.w, cnt[4 * j + 1] = b.z, cnt[4 * j + 2] = b.y, cnt[4 * j + 3] = b.x;
      c += b.x + b.y + b.z + b.w;
    }
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
    if (open > 0 && count <= kNearKeys && count <= NT) {
      for_keys<NT, T>(key4, n, tid, [&](int, T k) {
        if ((k ^ base) >> open == 0) {
          const int at = atomicAdd(&sm.filled, 1);
          if (at < kNearKeys) sm.near_[at] = k;
        }
      });
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

// (key1(i): one of them.)  Calls emit(position, i, key) for every key above t, and for the first need of
// those equal to t, in increasing order of i, at most `room` of them (keys that
// another launch overwrites meanwhile must not write past the list).  Whole
// CTA: every warp counts its consecutive stretch, then lists it.
template <int NT, class T, class Key4, class Key1, class Emit>
__device__ void take_above(Key4 key4, Key1 key1, int n, T t, int need, int room, SelectSmem<NT> &sm, int tid, Emit emit) {
  const int lane = tid & 31, warp = tid >> 5;
  const int seg = (n + 4 * NT - 1) / (4 * NT) * 128;  // keys of a warp
  const int beg = min(n, warp * seg), end = min(n, beg + seg);
  int gt = 0, eq = 0;
#pragma unroll 2
  for (int i = beg + 4 * lane; i < end; i += 128) {
    const Keys4<T> k = key4(i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      gt += i + e < end && k.v[e] > t;
      eq += i + e < end && k.v[e] == t;
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  __syncthreads();
  if (lane == 0) {
    sm.a[warp] = gt;
    sm.b[warp] = eq;
  }
  __syncthreads();
  gt = eq = 0;
  int all_eq = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) {
      gt += sm.a[w];
      eq += sm.b[w];
    }
    all_eq += sm.b[w];
  }
  const bool every = need >= all_eq;  // then the order of the equal ones does not matter
  const unsigned int below = (1u << lane) - 1u;
  int pos = gt + min(eq, need);
#pragma unroll 4
  for (int i0 = beg; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    const T k = i < end ? key1(i) : (T)0;
    bool in = i < end && (k > t || (every && k == t));
    if (!every) {
      const unsigned int same = __ballot_sync(0xffffffffu, i < end && k == t);
      in |= (same >> lane & 1u) && eq + __popc(same & below) < need;
      eq += __popc(same);
    }
    const unsigned int b = __ballot_sync(0xffffffffu, in);
    const int at = pos + __popc(b & below);
    if (in && at < room) emit(at, i, k);
    pos += __popc(b);
  }
}

}  // namespace
}  // namespace pa
