// Device-side helpers of the operators around the recurrence: element-aligned
// vector loads, exchanges inside rows of 16 lanes, and the activations.
#pragma once

#include "kda_device.h"
#include "kda_layer.h"
#include "kda_seqs.h"

namespace kda {

// ---- vectors ---------------------------------------------------------------
// V consecutive elements as floats.  Slices start at any element, so the
// vector types carry the alignment of one element only (the hardware takes
// such addresses).
template <typename T, int V> struct Pack {
  typedef T type __attribute__((ext_vector_type(V), aligned(sizeof(T))));
};
template <typename T> struct Pack<T, 1> {
  typedef T type;
};

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[V]) {
  const typename Pack<T, V>::type r = *(const typename Pack<T, V>::type*)p;
  if constexpr (V == 1) {
    v[0] = Elem<T>::to_f32(r);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = Elem<T>::to_f32(r[i]);
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = Elem<T>::from_f32(v[0]);
  } else if constexpr (sizeof(T) == 2) {
    typedef uint32_t words __attribute__((ext_vector_type(V / 2), aligned(2)));
    words r;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r[i] = __builtin_bit_cast(uint32_t, f32x2_to_bf16x2(v[2 * i], v[2 * i + 1]));
    *(words*)p = r;
  } else {
    typename Pack<T, V>::type r;
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = v[i];
    *(typename Pack<T, V>::type*)p = r;
  }
}
template <typename T>
__device__ __forceinline__ float load_f32(const T* p) {
  return Elem<T>::to_f32(*p);
}

// A value that every lane of the wave holds alike, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// ---- rows of 16 lanes --------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// lane K's value in every lane of its row
template <int K>
__device__ __forceinline__ float row_bcast(float v) {
  return dpp<0x150 + K>(v);
}
constexpr int kRowMirror = 0x140, kHalfMirror = 0x141, kQuadMirror = 0x1b, kPairSwap = 0xb1, kQuadSwap = 0x4e,
              kRotate4 = 0x124, kRotate8 = 0x128;

// sum over the row, in every lane
__device__ __forceinline__ float row_sum(float v) {
  v += dpp<kPairSwap>(v);
  v += dpp<kQuadMirror>(v);
  v += dpp<kHalfMirror>(v);
  v += dpp<kRowMirror>(v);
  return v;
}

// calls f(std::integral_constant<int, 0>) .. f(<N - 1>)
template <typename F, int... I>
__device__ __forceinline__ void static_for(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for(static_cast<F&&>(f), std::make_integer_sequence<int, N>{});
}

// ---- activations -------------------------------------------------------------
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.f + exp2_fast(-kLog2e * v));
}
// log(1 + e^v): max(v, 0) + log1p(u) with u = e^-|v| in (0, 1]; the second
// term of log1p(u) = log(w) + (u - (w - 1)) is what rounding w = 1 + u lost.
__device__ __forceinline__ float softplus(float v) {
  const float u = exp2_fast(-kLog2e * __builtin_fabsf(v));
  const float w = 1.f + u;
  return fmaxf(v, 0.f) + (kLn2 * __builtin_amdgcn_logf(w) + (u - (w - 1.f)));
}

}  // namespace kda
