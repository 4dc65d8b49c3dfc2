// Activations, rows of them in vectors of VEC elements, and sums over the threads
// of a workgroup that hold a row.
#pragma once

#include "mfma_ops.h"

namespace ckda {

template <class IO>
__device__ __forceinline__ float sigmoid_of(float x) {
  // off by 1e-6 of the value at most in the fast form, far below bf16's rounding
  if constexpr (sizeof(typename IO::storage) == 2)
    return __builtin_amdgcn_rcpf(1.f + exp_neg(x));
  else
    return 1.f / (1.f + expf(-x));
}

// sigmoid p and its derivative q = e p^2, e = exp(-x): p (1 - p) would lose the
// digits of q where p is next to 1 (a percent at 12, all of it from 17 on).
// Where e overflows p is 0, and so is q.
template <class IO>
__device__ __forceinline__ void sigmoid_and_slope(float x, float& p, float& q) {
  float e;
  if constexpr (sizeof(typename IO::storage) == 2) {
    e = exp_neg(x);
    p = __builtin_amdgcn_rcpf(1.f + e);
  } else {
    e = expf(-x);
    p = 1.f / (1.f + e);
  }
  q = p == 0.f ? 0.f : e * p * p;
}

// silu and its slope; zeros where the sigmoid is (also at -inf)
template <class IO>
__device__ __forceinline__ float silu_of(float x) {
  const float p = sigmoid_of<IO>(x);
  return p == 0.f ? 0.f : x * p;
}
template <class IO>
__device__ __forceinline__ void silu_and_slope(float x, float& y, float& s) {
  float p, q;
  sigmoid_and_slope<IO>(x, p, q);
  y = p == 0.f ? 0.f : x * p;
  s = p == 0.f ? 0.f : p + (q == 0.f ? 0.f : x * q);
}

// VEC elements at p (aligned to VEC elements), widened
template <class IO, int VEC>
struct Vec {
  using T = typename IO::storage;
  typedef T V __attribute__((ext_vector_type(VEC)));
  static __device__ __forceinline__ V load(const void* p, int64_t i) {
    return __builtin_nontemporal_load(reinterpret_cast<const V*>(static_cast<const T*>(p) + i));
  }
  static __device__ __forceinline__ float get(const V& v, int e) {
    T x;
    if constexpr (VEC == 1)
      x = v[0];
    else
      x = v[e];
    if constexpr (sizeof(T) == 2)
      return bf16_to_f32(x);
    else
      return x;
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float* x) {
    V v;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if constexpr (sizeof(T) == 2) {
        const __bf16 b = static_cast<__bf16>(x[e]);
        v[e] = __builtin_bit_cast(uint16_t, b);
      } else {
        v[e] = x[e];
      }
    }
    __builtin_nontemporal_store(v, reinterpret_cast<V*>(static_cast<T*>(p) + i));
  }
};

// VEC elements of a row.  ALIGNED: whole vectors at multiples of their size,
// streamed.  Otherwise they may lie anywhere and the row's last one may hold fewer
// (n elements): wide accesses all the same, which the memory path splits where they
// cross a line, and cached ones, since neighbours share lines.  Measured on 40000
// rows of 1001 float32: a convolution takes 67 us so, 128 an element at a time.
template <class IO, int VEC, bool ALIGNED>
struct Chans {
  using T = typename IO::storage;
  typedef T V __attribute__((ext_vector_type(VEC)));
  struct __attribute__((packed)) Any {
    T x[VEC];
  };
  static __device__ __forceinline__ V load(const void* p, int64_t i, int n) {
    const T* at = static_cast<const T*>(p) + i;
    if constexpr (ALIGNED) return __builtin_nontemporal_load(reinterpret_cast<const V*>(at));
    V v = V{};
    if (n >= VEC) {
      const Any a = *reinterpret_cast<const Any*>(at);
      v = __builtin_bit_cast(V, a);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e < n) v[e] = at[e];
    }
    return v;
  }
  static __device__ __forceinline__ float get(const V& v, int e) {
    if constexpr (sizeof(T) == 2)
      return bf16_to_f32(v[e]);
    else
      return v[e];
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, int n, const float* x) {
    T* at = static_cast<T*>(p) + i;
    V v;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if constexpr (sizeof(T) == 2)
        v[e] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x[e]));
      else
        v[e] = x[e];
    }
    if constexpr (ALIGNED) {
      __builtin_nontemporal_store(v, reinterpret_cast<V*>(at));
    } else if (n >= VEC) {
      *reinterpret_cast<Any*>(at) = __builtin_bit_cast(Any, v);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e < n) at[e] = v[e];
    }
  }
  // widened
  static __device__ __forceinline__ void row(const void* p, int64_t i, int n, float* x) {
    const V v = load(p, i, n);
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = get(v, e);
  }
};

// Sums of N values over the TPR threads of a row (a power of two); `red` holds
// 2 * MOST floats a wave and is used alternately (two halves), so one barrier a sum.
template <int N, int NT, int MOST = 2>
__device__ __forceinline__ void row_sum(float (&v)[N], int tpr, float* red, int& half) {
  const int wide = tpr < 64 ? tpr : 64;
  for (int m = wide >> 1; m >= 1; m >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], m, 64);
  if (tpr <= 64) return;
  const int t = threadIdx.x, wave = t >> 6, waves = tpr >> 6;
  float* r = red + half * (NT / 64) * MOST;
  half ^= 1;
  if ((t & 63) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) r[MOST * wave + i] = v[i];
  __syncthreads();
  // the row's waves are the whole workgroup (tpr = NT) or an aligned part of it
  const int first = wave & ~(waves - 1);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  // two waves' at a time: the compiler's eight hold 8 N registers at the kernels' tightest
  // place (gradients of 4096 rows of 16384 in bf16: block norm 5956 us against 1128 so;
  // layer norm, with a sum more, 421 against 366 at 16383 elements)
#pragma unroll 2
  for (int j = 0; j < waves; ++j)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += r[MOST * (first + j) + i];
}

}  // namespace ckda
