// Vectors of activations in fp32 or bf16.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>

namespace gdn {

// V neighbouring elements, moved as one access of up to 16 bytes (two or more
// for larger ones).
template <typename T, int V>
struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Vec {
  T v[V];
};

// V fp32 values worked on together; pairs by the packed instructions (one for
// two multiply-adds, each rounded as the scalar one).
template <int V>
struct alignas(4 * V) F {
  float v[V];
};

__device__ __forceinline__ uint64_t bits(F<2> a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.v[0]), "f"(a.v[1]));
  return r;
}
__device__ __forceinline__ F<2> pair(uint64_t r) {
  F<2> a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.v[0]), "=f"(a.v[1]) : "l"(r));
  return a;
}
__device__ __forceinline__ F<2> fma(F<2> a, F<2> b, F<2> c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return pair(r);
}
__device__ __forceinline__ F<2> mul(F<2> a, F<2> b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return pair(r);
}
__device__ __forceinline__ F<2> add(F<2> a, F<2> b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return pair(r);
}
template <int V>
__device__ __forceinline__ F<V> all(float x) {
  F<V> r;
#pragma unroll
  for (int e = 0; e < V; ++e) r.v[e] = x;
  return r;
}
__device__ __forceinline__ F<1> fma(F<1> a, F<1> b, F<1> c) { return {{fmaf(a.v[0], b.v[0], c.v[0])}}; }
__device__ __forceinline__ F<1> mul(F<1> a, F<1> b) { return {{a.v[0] * b.v[0]}}; }
__device__ __forceinline__ F<1> add(F<1> a, F<1> b) { return {{a.v[0] + b.v[0]}}; }

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16(x);  // nearest even: the one rounding of a result
}

template <int V>
__device__ __forceinline__ F<V> to_f(const Vec<float, V>& x) {
  F<V> r;
#pragma unroll
  for (int e = 0; e < V; ++e) r.v[e] = x.v[e];
  return r;
}
template <int V>
__device__ __forceinline__ F<V> to_f(const Vec<__nv_bfloat16, V>& x) {
  F<V> r;
#pragma unroll
  for (int e = 0; e < V; ++e) r.v[e] = to_f(x.v[e]);
  return r;
}

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load(const T* p) {
  return *reinterpret_cast<const Vec<T, V>*>(p);
}
// Starts an asynchronous copy of one E (4, 8 or 16 bytes) to shared memory.
template <typename E>
__device__ __forceinline__ void copy_async(E* dst, const E* src) {
  const unsigned d = static_cast<unsigned>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(sizeof(E))
               : "memory");
}
// The same, or zeros (bytes 0; nothing is read then).
template <typename E>
__device__ __forceinline__ void copy_async(E* dst, const E* src, int bytes) {
  const unsigned d = static_cast<unsigned>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(src),
               "n"(sizeof(E)), "r"(bytes)
               : "memory");
}

template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float (&x)[V]) {
  Vec<T, V> r;
#pragma unroll
  for (int e = 0; e < V; ++e) r.v[e] = from_f<T>(x[e]);
  *reinterpret_cast<Vec<T, V>*>(p) = r;
}

}  // namespace gdn
