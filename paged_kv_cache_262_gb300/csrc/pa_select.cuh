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

// Sum of v[0 .. warp - 1], a value a warp of the CTA.
template <int NT>
__device__ __forceinline__ int sum_before(const int *v, int lane, int warp) {
  return __reduce_add_sync(0xffffffffu, lane < warp && lane < NT / 32 ? v[lane] : 0);
}
template <int NT>
__device__ __forceinline__ int sum_all(const int *v, int lane) {
  return __reduce_add_sync(0xffffffffu, lane < NT / 32 ? v[lane] : 0);
}

// f(i, key) for every key of this thread: four consecutive ones at a time.
template <int NT, class T, class Key4, class F>
__device__ __forceinline__ void for_keys(Key4 key4, int n, int tid, F f) {
#pragma unroll 4
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
  lo = (T)sm.lo[lane % (NT / 32)];
  hi = (T)sm.hi[lane % (NT / 32)];
#pragma unroll
  for (int o = NT / 64; o > 0; o >>= 1) {
    const T l2 = __shfl_xor_sync(0xffffffffu, lo, o), h2 = __shfl_xor_sync(0xffffffffu, hi, o);
    lo = l2 < lo ? l2 : lo;
    hi = h2 > hi ? h2 : hi;
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
    int run = incl - c + sum_before<NT>(sm.a, lane, warp);
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

// The same for n <= NT keys, a thread a key: the least key that fewer than want
// are above (300 instructions and two barriers where the bins take 1.5 us).
template <int NT, class T, class Key4, class Key1>
__device__ Kth<T> kth_of_few(Key4 key4, Key1 key1, int n, int want, SelectSmem<NT> &sm, int tid) {
  static_assert(sizeof(T) == 4, "32-bit keys");
  const T mine = tid < n ? key1(tid) : (T)0;
  int gt = 0;
#pragma unroll 4
  for (int j = 0; j + 4 <= n; j += 4) {
    const Keys4<T> k = key4(j);
#pragma unroll
    for (int e = 0; e < 4; ++e) gt += k.v[e] > mine;
  }
  for (int j = n & ~3; j < n; ++j) gt += key1(j) > mine;
  T t = __reduce_min_sync(0xffffffffu, tid < n && gt < want ? mine : ~(T)0);
  const int lane = tid & 31;
  __syncthreads();  // sm may be in use by a call before
  if (lane == 0) sm.lo[tid >> 5] = t;
  __syncthreads();
  t = __reduce_min_sync(0xffffffffu, lane < NT / 32 ? (T)sm.lo[lane] : ~(T)0);
  if (tid < n && mine == t) sm.kth_above = gt;  // (equal keys write the same)
  __syncthreads();
  return Kth<T>{t, sm.kth_above};
}

// A warp's stretch of consecutive keys when the CTA's warps share n of them.
template <int NT>
struct Stretch {
  int beg, end;
  __device__ Stretch(int n, int warp) {
    const int seg = (n + 4 * NT - 1) / (4 * NT) * 128;
    beg = min(n, warp * seg);
    end = min(n, beg + seg);
  }
};

// Calls emit(position, i, key) for the keys of the warp's stretch that are at
// least t (eq_before + those equal to t before them < need, unless `every`
// equal one is taken), in increasing order of i, from position pos on and below
// `room` (keys that another launch overwrites meanwhile must not write past the
// list).  key1(i): a key.
template <int NT, class T, class Key1, class Emit>
__device__ __forceinline__ void list_stretch(Key1 key1, Stretch<NT> w, T t, bool every, int eq_before, int need,
                                             int pos, int room, int lane, Emit emit) {
  const unsigned int below = (1u << lane) - 1u;
  if (every) {
#pragma unroll 4
    for (int i0 = w.beg; i0 < w.end; i0 += 32) {
      const int i = i0 + lane;
      const T k = i < w.end ? key1(i) : (T)0;
      const bool in = i < w.end && k >= t;
      const unsigned int b = __ballot_sync(0xffffffffu, in);
      const int at = pos + __popc(b & below);
      if (in && at < room) emit(at, i, k);
      pos += __popc(b);
    }
    return;
  }
  for (int i0 = w.beg; i0 < w.end; i0 += 32) {
    const int i = i0 + lane;
    const T k = i < w.end ? key1(i) : (T)0;
    const unsigned int same = __ballot_sync(0xffffffffu, i < w.end && k == t);
    const bool in = i < w.end && (k > t || (k == t && eq_before + __popc(same & below) < need));
    const unsigned int b = __ballot_sync(0xffffffffu, in);
    const int at = pos + __popc(b & below);
    if (in && at < room) emit(at, i, k);
    pos += __popc(b);
    eq_before += __popc(same);
  }
}

// The same over the whole CTA: emit for every key above t, and for the first
// need of those equal to t.
template <int NT, class T, class Key4, class Key1, class Emit>
__device__ void take_above(Key4 key4, Key1 key1, int n, T t, int need, int room, SelectSmem<NT> &sm, int tid,
                           Emit emit) {
  const int lane = tid & 31, warp = tid >> 5;
  const Stretch<NT> w(n, warp);
  int gt = 0, eq = 0;
#pragma unroll 4
  for (int i = w.beg + 4 * lane; i < w.end; i += 128) {
    const Keys4<T> k = key4(i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      gt += i + e < w.end && k.v[e] > t;
      eq += i + e < w.end && k.v[e] == t;
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
  gt = sum_before<NT>(sm.a, lane, warp);
  eq = sum_before<NT>(sm.b, lane, warp);
  const bool every = need >= sum_all<NT>(sm.b, lane);  // then the order of the equal ones does not matter
  list_stretch<NT, T>(key1, w, t, every, eq, need, gt + min(eq, need), room, lane, emit);
}

}  // namespace
}  // namespace pa
