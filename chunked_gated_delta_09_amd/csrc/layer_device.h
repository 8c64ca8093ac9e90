// Device-side helpers shared by the layer operators' kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer_launch.h"

namespace kda {

typedef __bf16 bf16;

__device__ __forceinline__ float as_f(bf16 x) { return (float)x; }
__device__ __forceinline__ float as_f(float x) { return x; }

// N elements as loaded, in whole registers: two bf16 each (elements of their own would take a
// register each wherever two ways of loading them meet).
template <class T, int N>
struct Pack {
  static constexpr int WORDS = (N * (int)sizeof(T) + 3) / 4;
  uint32_t w[WORDS];
  __device__ __forceinline__ float at(int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    return __uint_as_float(e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  }
  // sets an element of a Pack of zeros
  __device__ __forceinline__ void put(int e, T x) {
    if constexpr (sizeof(T) == 4)
      w[e] = __builtin_bit_cast(uint32_t, x);
    else
      w[e / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, x) << (16 * (e % 2));
  }
};

// N elements at p; those from `valid` on are zero. `vec`: p is aligned for one load of all N.
template <class T, int N>
__device__ __forceinline__ Pack<T, N> load_n(const T* p, int valid, bool vec) {
  Pack<T, N> r;
  if (vec && valid >= N && N > 1) {
    struct alignas(sizeof(T) * N < 4 ? 4 : sizeof(T) * N) Words {
      uint32_t w[Pack<T, N>::WORDS];
    };
    const Words v = *reinterpret_cast<const Words*>(p);
#pragma unroll
    for (int i = 0; i < Pack<T, N>::WORDS; ++i) r.w[i] = v.w[i];
  } else {
#pragma unroll
    for (int i = 0; i < Pack<T, N>::WORDS; ++i) r.w[i] = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < valid) r.put(i, p[i]);
  }
  return r;
}

// N values to p, rounded to T; those from `valid` on are left. The wide and the single stores take different
// words, or the compiler joins the two ways into one of single stores.
template <class T, int N>
__device__ __forceinline__ void store_n(T* p, const float (&x)[N], int valid, bool vec) {
  if (vec && valid >= N && N > 1) {
    struct alignas(sizeof(T) * N < 4 ? 4 : sizeof(T) * N) Words {
      uint32_t w[Pack<T, N>::WORDS];
    } r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) r.w[i] = __float_as_uint(x[i]);
    } else {
      typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
      for (int i = 0; i + 1 < N; i += 2) {
        const bf16x2 v = {(bf16)x[i], (bf16)x[i + 1]};
        r.w[i / 2] = __builtin_bit_cast(uint32_t, v);
      }
    }
    *reinterpret_cast<Words*>(p) = r;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < valid) p[i] = (T)x[i];
  }
}

// Four fp32 values of a state that a token step passes through once: past the caches, which hold
// nothing of it by the next step. On the KDA step of 256 sequences x 32 heads of 128 x 128 (1.07 GB in
// place) 210 us, against 233 through them; the scan's of 128 sequences (67 MB) 19.5 against 20.5; one sequence of
// 16 heads takes 4.9 us either way.
__device__ __forceinline__ float4 load_stream(const float* p) {
  typedef float f4 __attribute__((ext_vector_type(4)));
  const f4 v = __builtin_nontemporal_load(reinterpret_cast<const f4*>(p));
  return make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_stream(float* p, float4 v) {
  typedef float f4 __attribute__((ext_vector_type(4)));
  const f4 w = {v.x, v.y, v.z, v.w};
  __builtin_nontemporal_store(w, reinterpret_cast<f4*>(p));
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// 2^x by the hardware instruction (results below the normal range become zero).
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
// 1 / (1 + e^-x): e^-x overflows to infinity for x < -88.7, where the quotient is zero as it should be.
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + exp2_hw(-kLog2e * x)); }
// log(1 + e^x) = max(x, 0) + log1p(e^-|x|): no overflow, and full relative precision for very
// negative x, where it is e^x. With u = 1 + e rounded, log1p(e) is log(u) + (e - (u - 1)) / u; u is in
// [1, 2], so the hardware's log2 needs none of a general logarithm's scaling.
__device__ __forceinline__ float softplus(float x) {
  const float e = exp2_hw(-kLog2e * fabsf(x));
  const float u = 1.f + e;
  float top;  // one instruction; fmaxf is two, the first for signalling NaN
  asm("v_max_f32 %0, 0, %1" : "=v"(top) : "v"(x));
  return fmaf(__builtin_amdgcn_logf(u), kLn2, fmaf(e - (u - 1.f), __builtin_amdgcn_rcpf(u), top));
}

// The derivative of x sigmoid(x).
__device__ __forceinline__ float dsilu(float x) {
  const float s = sigmoid(x);
  return s * (1.f + x * (1.f - s));
}

// Moves within rows of 16 lanes (DPP controls): quad permutations, mirrors, rotations, shifts.
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kRor8 = 0x128, kShl4 = 0x104;
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  const int v = __float_as_int(x);
  return __int_as_float(__builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, true));
}
// x + the value of the lane that differs in bit 4 (bit 5).
__device__ __forceinline__ float add_xor16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float add_xor32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sum over the L lanes of an aligned group (L a power of two), in every lane. The mirror of 8 lanes
// stands for the lane 4 away: the four lanes of a quad hold the same sum by then.
template <int L>
__device__ __forceinline__ float group_sum(float x) {
  if constexpr (L >= 2) x += dpp<kXor1>(x);
  if constexpr (L >= 4) x += dpp<kXor2>(x);
  if constexpr (L >= 8) x += dpp<kHalfMirror>(x);
  if constexpr (L >= 16) x += dpp<kRor8>(x);
  if constexpr (L >= 32) x = add_xor16(x);
  if constexpr (L >= 64) x = add_xor32(x);
  return x;
}

// The sequence that holds token t: the last n with first(n) <= t, over a table of n + 1 firsts.
__device__ __forceinline__ int find_seq(const int32_t* first, int n, int64_t t) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ int64_t seq_begin(const Seqs& s, int n) { return s.cu ? s.cu[n] : (int64_t)n * s.T; }
__device__ __forceinline__ int64_t seq_end(const Seqs& s, int n) { return s.cu ? s.cu[n + 1] : (int64_t)(n + 1) * s.T; }
__device__ __forceinline__ int seq_of(const Seqs& s, int64_t t) {
  return s.cu ? find_seq(s.cu, s.n, t) : (int)((uint32_t)t / (uint32_t)s.T);  // tokens fit 31 bits
}

// The state row of batch row b in a token step: slots[b], or b itself without a table. A negative slot
// is a padding row (-1); a slot behind the last row, or one that an earlier batch row has already, is
// refused (-2): the first batch row owns it, and two rows never write the same state. The whole
// workgroup calls it.
__device__ __forceinline__ int step_slot(const int32_t* slots, int b, int n) {
  if (slots == nullptr) return b;
  const int s = slots[b];
  int seen = 0;
  for (int i = threadIdx.x; i < b; i += blockDim.x) seen |= slots[i] == s;
  seen = __syncthreads_or(seen);
  if (s < 0) return -1;
  return s >= n || seen ? -2 : s;
}

}  // namespace kda
