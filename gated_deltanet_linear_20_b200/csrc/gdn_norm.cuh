// What the norm kernels share: the layout of a row over threads, its sums, the
// gate, and the choice of a layout.
//
// A row of D channels is held in registers by `threads per row` threads, NV
// vectors of V channels each (vector j of thread t: channels (j TPR + t) V ..),
// so it is read from memory once, whatever is summed over it.  Sub-warp rows
// (TPR 8, 16, 32) share a CTA and sum by shuffles; longer ones have a CTA.
#pragma once

#include <algorithm>

#include "gdn_internal.h"
#include "gdn_vec.cuh"

namespace gdn {

constexpr int kNormThreads = 256;     // of a CTA of sub-warp rows
constexpr int kNormMaxThreads = 512;  // of a CTA with one row

// Sums of K values over the threads of a row; every thread gets them.  TPR == 0:
// the row is the whole CTA's.  `buf` holds two sets, used in turn, so that one
// barrier a sum is enough; the order of the additions is fixed.
template <int TPR, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*buf)[K][16], int& turn) {
  constexpr int W = TPR == 0 ? 32 : TPR;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (TPR == 0) {
    const int w = threadIdx.x >> 5, n = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) buf[turn][k][w] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = 0.f;
      for (int i = 0; i < n; ++i) v[k] += buf[turn][k][i];
    }
    turn ^= 1;
  }
}

// The gate's value and slope.  1 / (1 + exp(-z)) from the approximate exponential
// and quotient: a few units in the last place of fp32.
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }
__device__ __forceinline__ float gate(int act, float z) {
  const float p = sigmoid(z);
  return act == GDN_GATE_SILU ? z * p : p;
}
__device__ __forceinline__ void gate_slope(int act, float z, float* a, float* da) {
  const float p = sigmoid(z);
  *a = act == GDN_GATE_SILU ? z * p : p;
  *da = act == GDN_GATE_SILU ? p * (1.f + z * (1.f - p)) : p * (1.f - p);
}

template <typename T, int V, int NV>
__device__ __forceinline__ void load_row(Vec<T, V> (&r)[NV], const T* p, int t, int tpr, int D) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * tpr + t) * V;
    if (c < D) {
      r[j] = load<T, V>(p + c);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) r[j].v[e] = from_f<T>(0.f);
    }
  }
}

// The weights of this thread's channels, `offset` added; `fill` without any.
template <int V, int NV>
__device__ __forceinline__ void load_weight(float (&w)[NV][V], const float* p, float offset,
                                            float fill, int t, int tpr, int D) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * tpr + t) * V;
    if (p && c < D) {
      const Vec<float, V> v = load<float, V>(p + c);
#pragma unroll
      for (int e = 0; e < V; ++e) w[j][e] = v.v[e] + offset;
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) w[j][e] = p ? 0.f : fill;
    }
  }
}

template <typename T, int V, int NV>
__device__ __forceinline__ void store_row(T* p, const float (&x)[NV][V], int t, int tpr, int D) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * tpr + t) * V;
    if (c < D) store<T, V>(p + c, x[j]);
  }
}

// A CTA's partial sums of one weight gradient, one row of D values: the CTA's
// rows_per_cta groups are added in order through shared memory.
template <int TPR, int V, int NV>
__device__ __forceinline__ void store_partial(float* part, const float (&acc)[NV][V], float* smem,
                                              int t, int tpr, int D) {
  if constexpr (TPR == 0) {
    store_row<float, V, NV>(part, acc, t, tpr, D);
  } else {
    const int group = threadIdx.x / TPR, groups = kNormThreads / TPR;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e)
        smem[group * (TPR * NV * V) + (j * TPR + t) * V + e] = acc[j][e];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kNormThreads) {
      float s = 0.f;
      for (int i = 0; i < groups; ++i) s += smem[i * (TPR * NV * V) + c];
      part[c] = s;
    }
  }
}

// Calls f.template run<TPR, NV, V>() with the layout for rows of D channels:
// 16-byte accesses where D is a multiple of 8 and every array starts on 16
// bytes (`wide`), else single elements.  TPR 0: one CTA a row.
template <typename F>
int with_layout(int D, bool wide, F&& f) {
  if (wide && D % 8 == 0) {
    if (D <= 64) return f.template run<8, 1, 8>();
    if (D <= 128) return f.template run<16, 1, 8>();
    if (D <= 256) return f.template run<32, 1, 8>();
    if (D <= 8 * kNormMaxThreads) return f.template run<0, 1, 8>();
    if (D <= 16 * kNormMaxThreads) return f.template run<0, 2, 8>();
    return f.template run<0, 4, 8>();
  }
  if (D <= 256) return f.template run<32, 8, 1>();
  if (D <= 8 * kNormMaxThreads) return f.template run<0, 8, 1>();
  return f.template run<0, 32, 1>();
}

// Threads of a CTA in the layout <TPR, NV, V>.
template <int TPR, int NV, int V>
int norm_threads(int D) {
  if (TPR > 0) return kNormThreads;
  const int need = (D + NV * V - 1) / (NV * V);
  return (need + 31) / 32 * 32;
}

// dst[i] = sum over parts p < n of part[p][i], i < cols.
int launch_reduce_parts(const float* part, int n, int cols, float* const* dst, int D,
                        cudaStream_t stream);

}  // namespace gdn
