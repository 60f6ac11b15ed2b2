// What the norm kernels share: the layout of a row over threads, its sums, the
// gate, and the choice of a layout.
//
// A row of D channels is held in registers by `threads per row` threads, NV
// vectors of V channels each (vector j of thread t: channels (j TPR + t) V ..),
// so it is read from memory once, whatever is summed over it.  Sub-warp rows
// (TPR 8, 16, 32) share a CTA and sum by shuffles; longer ones have a CTA.
//
// CTAs are persistent, and each thread copies its part of the next rows to shared
// memory asynchronously (a ring of two or three stages) while it works on the present one:
// the sums over a row and their barriers would leave the memory idle otherwise.
// A thread reads only what it copied, so the ring needs no barrier.
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

// Stages of a ring whose arrays have `bytes` a channel in all: three, if the
// longest staged row leaves room for them.
constexpr int stages(size_t bytes) { return bytes * 8 * kNormMaxThreads * 3 <= 220 * 1024 ? 3 : 2; }
// Staged layouts: vectors of four (cp.async moves at least 4 bytes), up to two a
// thread (larger rows would not fit the ring).
template <int NV, int V>
constexpr bool kStaged = V == 4 && NV <= 2;

// The ring of one array: NV vectors of each thread in each stage.
template <typename T, int V, int NV, int kStages>
struct Ring {
  Vec<T, V>* at;
  __device__ __forceinline__ Ring(unsigned char*& smem) : at(reinterpret_cast<Vec<T, V>*>(smem)) {
    smem += sizeof(Vec<T, V>) * NV * kStages * blockDim.x;
  }
  __device__ __forceinline__ Vec<T, V>* slot(int stage, int j) const {
    return at + (stage * NV + j) * blockDim.x + threadIdx.x;
  }
  // channels c >= D are zeros (D = 0: all of them, nothing is read)
  __device__ __forceinline__ void fetch(int stage, const T* p, int t, int tpr, int D) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * tpr + t) * V;
      copy_async(slot(stage, j), reinterpret_cast<const Vec<T, V>*>(c < D ? p + c : p),
                 c < D ? int(sizeof(Vec<T, V>)) : 0);
    }
  }
  __device__ __forceinline__ void take(Vec<T, V> (&r)[NV], int stage) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) r[j] = *slot(stage, j);
  }
};
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kStages>
__device__ __forceinline__ void copies_wait() {  // for the oldest stage in flight
  asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
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
// vectors of four where D is a multiple of 4 and every array starts on one
// (`wide`: 8 bytes of bf16, 16 of fp32), else single elements.  TPR 0: one CTA a
// row.
template <typename F>
int with_layout(int D, bool wide, F&& f) {
  if (wide && D % 4 == 0) {
    if (D <= 64) return f.template run<8, 2, 4>();
    if (D <= 128) return f.template run<16, 2, 4>();
    if (D <= 256) return f.template run<32, 2, 4>();
    if (D <= 8 * kNormMaxThreads) return f.template run<0, 2, 4>();
    if (D <= 16 * kNormMaxThreads) return f.template run<0, 4, 4>();
    return f.template run<0, 8, 4>();
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
