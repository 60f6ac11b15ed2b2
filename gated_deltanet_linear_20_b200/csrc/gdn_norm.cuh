// What the norm kernels share: the layout of a row over threads, its sums, the
// gate, and the copies of the next rows.
//
// A row of D channels is held in registers by TPR threads, NV vectors of V
// channels each (vector j of thread t: channels (j TPR + t) V ..), so it is read
// from memory once, whatever is summed over it.  Short rows (TPR 8, 16, 32)
// share a CTA of TH threads and sum by shuffles; longer ones have a CTA
// (TPR == TH).
//
// CTAs are persistent, and each thread copies its part of the next rows to shared
// memory asynchronously (a ring of two or three stages) while it works on the
// present one: the sums over a row and their barriers would leave the memory
// idle otherwise.  A thread reads only what it copied, so the ring needs no
// barrier.  What is left is the instruction count, so that all sizes of a layout
// are constants and channels are worked on in pairs.
#pragma once

#include <algorithm>

#include "gdn_host.h"
#include "gdn_internal.h"
#include "gdn_vec.cuh"

namespace gdn {

template <int TPR_, int TH_, int NV_, int V_>
struct Layout {
  static constexpr int TPR = TPR_, TH = TH_, NV = NV_, V = V_;
  static constexpr bool kShort = TPR <= 32;   // several rows a CTA
  static constexpr int kRows = TH / TPR;
  static constexpr int P = V >= 2 ? 2 : 1;    // channels worked on together
  static constexpr int N = NV * V / P;        // such groups of a thread
  // cp.async moves at least 4 bytes, and longer rows would not fit the ring
  static constexpr bool kStaged = V == 4 && NV * TH <= 1024;
};

// Stages of a ring whose arrays have `bytes` a channel in all: three, if the
// longest staged row leaves room for them.
constexpr int stages(size_t bytes) { return bytes * 4096 * 3 <= 220 * 1024 ? 3 : 2; }
template <typename L>
constexpr size_t ring_bytes(size_t bytes) {
  return L::kStaged ? stages(bytes) * bytes * L::TH * L::NV * L::V : 0;
}

// This thread's place: the channel of its vector j is t V + j TPR V.
template <typename L>
struct Place {
  int sub;          // its row among the CTA's
  unsigned c0, D;   // its first channel, the row's channels
  __device__ __forceinline__ explicit Place(int d)
      : sub(L::kShort ? threadIdx.x / L::TPR : 0), c0((threadIdx.x % L::TPR) * L::V), D(d) {}
  __device__ __forceinline__ bool has(int j) const { return c0 + j * L::TPR * L::V < D; }
};

// The channels of vector j among a thread's groups.
template <typename L, typename T>
__device__ __forceinline__ void spread(F<L::P> (&r)[L::N], const Vec<T, L::V>& x, int j) {
#pragma unroll
  for (int e = 0; e < L::V; ++e) r[(j * L::V + e) / L::P].v[e % L::P] = to_f(x.v[e]);
}

// One input array in the ring: BEFORE bytes a channel of other arrays lie before
// it in a stage of ALL bytes a channel.
template <typename L, typename T, int BEFORE, int ALL>
struct Ring {
  using E = Vec<T, L::V>;
  static constexpr int kCh = L::TH * L::NV * L::V;
  __device__ __forceinline__ static E* slot(unsigned char* smem, int stage, int j) {
    return reinterpret_cast<E*>(smem + stage * (ALL * kCh) + BEFORE * kCh) + j * L::TH +
           threadIdx.x;
  }
  // Channels past D stay zero in every stage.
  __device__ __forceinline__ static void clear(unsigned char* smem, const Place<L>& at) {
#pragma unroll
    for (int s = 0; s < stages(ALL); ++s)
#pragma unroll
      for (int j = 0; j < L::NV; ++j)
        if (!at.has(j)) *slot(smem, s, j) = E{};
  }
  // p: the row's first channel; a row past the end is zeros
  __device__ __forceinline__ static void fetch(unsigned char* smem, int stage, const T* p,
                                               const Place<L>& at, bool on) {
#pragma unroll
    for (int j = 0; j < L::NV; ++j)
      if (at.has(j)) {
        const E* src = reinterpret_cast<const E*>(p + (at.c0 + j * L::TPR * L::V));
        if (L::kShort)
          copy_async(slot(smem, stage, j), src, on ? int(sizeof(E)) : 0);
        else
          copy_async(slot(smem, stage, j), src);
      }
  }
  __device__ __forceinline__ static void take(F<L::P> (&r)[L::N], unsigned char* smem, int stage) {
#pragma unroll
    for (int j = 0; j < L::NV; ++j) spread<L, T>(r, *slot(smem, stage, j), j);
  }
};

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int STAGES>
__device__ __forceinline__ void copies_wait() {  // for the oldest stage in flight
  asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
}

// A row straight from memory (layouts that are not staged).
template <typename L, typename T>
__device__ __forceinline__ void load_row(F<L::P> (&r)[L::N], const T* p, const Place<L>& at,
                                         bool on) {
#pragma unroll
  for (int j = 0; j < L::NV; ++j) {
    Vec<T, L::V> x{};
    if (on && at.has(j)) x = load<T, L::V>(p + (at.c0 + j * L::TPR * L::V));
    spread<L, T>(r, x, j);
  }
}

template <typename L, typename T>
__device__ __forceinline__ void store_row(T* p, const F<L::P> (&r)[L::N], const Place<L>& at,
                                          bool on) {
#pragma unroll
  for (int j = 0; j < L::NV; ++j)
    if (on && at.has(j)) {
      float x[L::V];
#pragma unroll
      for (int e = 0; e < L::V; ++e) x[e] = r[(j * L::V + e) / L::P].v[e % L::P];
      store<T, L::V>(p + (at.c0 + j * L::TPR * L::V), x);
    }
}

// The weights of this thread's channels, `offset` added; ones without any.
template <typename L>
__device__ __forceinline__ void load_weight(F<L::P> (&w)[L::N], const float* p, float offset,
                                            const Place<L>& at) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < L::N; ++i) w[i] = all<L::P>(1.f);
    return;
  }
  load_row<L, float>(w, p, at, true);
#pragma unroll
  for (int i = 0; i < L::N; ++i) w[i] = add(w[i], all<L::P>(offset));
}

template <int P>
__device__ __forceinline__ float total(F<P> a) {
  return P == 2 ? a.v[0] + a.v[P - 1] : a.v[0];
}

// Sums of K values over the threads of a row; every thread gets them.  For rows
// of several warps `buf` holds two sets, used in turn, so that one barrier a sum
// is enough.  The order of the additions is fixed.
template <typename L, int K>
struct SumBuffer {
  static constexpr int kWarps = L::TH / 32;
  float part[2][K == 1 ? 1 : 4][kWarps];
};
template <typename L, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], SumBuffer<L, K>& buf, int& turn) {
  constexpr int n = L::TH / 32;
  const auto halve = [](float x, int o) { return x + __shfl_xor_sync(0xffffffffu, x, o); };
  if constexpr (L::kShort || K == 1) {
    constexpr int W = L::kShort ? L::TPR : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = halve(v[k], o);
    if constexpr (!L::kShort) {
      const int lane = threadIdx.x & 31;
      if (lane == 0) buf.part[turn][0][threadIdx.x >> 5] = v[0];
      __syncthreads();
      v[0] = buf.part[turn][0][lane % n];
#pragma unroll
      for (int o = n / 2; o > 0; o >>= 1) v[0] = halve(v[0], o);
      turn ^= 1;
    }
  } else {
    // up to four values at once: two exchanges leave value k with the lanes 8 k ..
    // 8 k + 7, so that the rest is one shuffle a step instead of K
    static_assert(K <= 4, "four groups of eight lanes");
    const int lane = threadIdx.x & 31, mine = lane >> 3;
    const bool hi = lane & 16, odd = lane & 8;
    const auto merge = [](bool second, float a, float b, int o) {
      return (second ? b : a) + __shfl_xor_sync(0xffffffffu, second ? a : b, o);
    };
    const float v1 = K > 1 ? v[K > 1 ? 1 : 0] : 0.f, v2 = K > 2 ? v[K > 2 ? 2 : 0] : 0.f,
                v3 = K > 3 ? v[K > 3 ? 3 : 0] : 0.f;
    float x = merge(odd, merge(hi, v[0], v2, 16), merge(hi, v1, v3, 16), 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) x = halve(x, o);
    if ((lane & 7) == 0) buf.part[turn][mine][threadIdx.x >> 5] = x;
    __syncthreads();
    x = buf.part[turn][mine][lane & (n < 8 ? n - 1 : 7)];
    if (n > 8) x += buf.part[turn][mine][(lane & 7) + (n > 8 ? 8 : 0)];
#pragma unroll
    for (int o = n < 8 ? n / 2 : 4; o > 0; o >>= 1) x = halve(x, o);
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, x, 8 * k);
    turn ^= 1;
  }
  static_assert(n == 4 || n == 8 || n == 16, "warps of a CTA");
}

// 1 / (1 + exp(-z)) from the approximate power and reciprocal: a few units in
// the last place of fp32; an overflowing exponential gives 0.
__device__ __forceinline__ float sigmoid(float z) {
  float e, p;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(1.f + e));
  return p;
}
// The gate's value and slope: p z and p (1 + z (1 - p)), or p and p (1 - p).
template <int P>
__device__ __forceinline__ F<P> gate(int act, F<P> z) {
  F<P> p;
#pragma unroll
  for (int e = 0; e < P; ++e) {
    p.v[e] = sigmoid(z.v[e]);
    z.v[e] = act == GDN_GATE_SILU ? z.v[e] : 1.f;
  }
  return mul(z, p);
}
template <int P>
__device__ __forceinline__ void gate_slope(int act, F<P> z, F<P>* a, F<P>* da) {
  F<P> p;
#pragma unroll
  for (int e = 0; e < P; ++e) {
    p.v[e] = sigmoid(z.v[e]);
    z.v[e] = act == GDN_GATE_SILU ? z.v[e] : 1.f;
  }
  const F<P> q = fma(p, all<P>(-1.f), all<P>(1.f));
  *a = mul(z, p);
  *da = mul(p, fma(z, q, all<P>(act == GDN_GATE_SILU ? 1.f : 0.f)));
}

// A CTA's partial sums of one weight gradient, one row of D values: its rows'
// groups of threads are added in order through shared memory.
template <typename L>
__device__ __forceinline__ void store_partial(float* part, const F<L::P> (&acc)[L::N], float* smem,
                                              const Place<L>& at) {
  if constexpr (L::kRows == 1) {
    store_row<L, float>(part, acc, at, true);
  } else {
    constexpr int kRow = L::TPR * L::NV * L::V;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < L::N; ++i)
#pragma unroll
      for (int e = 0; e < L::P; ++e) {
        const int k = i * L::P + e;
        smem[at.sub * kRow + at.c0 + (k / L::V) * L::TPR * L::V + k % L::V] = acc[i].v[e];
      }
    __syncthreads();
    for (unsigned c = threadIdx.x; c < at.D; c += L::TH) {
      float s = 0.f;
      for (int i = 0; i < L::kRows; ++i) s += smem[i * kRow + c];
      part[c] = s;
    }
  }
}

// Calls f.template run<Layout>() with the layout for rows of D channels: vectors
// of four where D is a multiple of 4 and every array starts on one (`wide`: 8
// bytes of bf16, 16 of fp32), else single elements.
template <typename F>
int with_layout(int D, bool wide, F&& f) {
  if (wide && D % 4 == 0) {
    if (D <= 64) return f.template run<Layout<8, 256, 2, 4>>();
    if (D <= 128) return f.template run<Layout<16, 256, 2, 4>>();
    if (D <= 256) return f.template run<Layout<32, 256, 2, 4>>();
    if (D <= 1024) return f.template run<Layout<128, 128, 2, 4>>();
    if (D <= 2048) return f.template run<Layout<256, 256, 2, 4>>();
    if (D <= 4096) return f.template run4096();
    if (D <= 8192) return f.template run<Layout<512, 512, 4, 4>>();
    return f.template run<Layout<512, 512, 8, 4>>();
  }
  if (D <= 256) return f.template run<Layout<32, 256, 8, 1>>();
  if (D <= 2048) return f.template run<Layout<256, 256, 8, 1>>();
  return f.template run<Layout<512, 512, 32, 1>>();
}

// dst[i] = sum over parts p < n of part[p][i], i < cols.
int launch_reduce_parts(const float* part, int n, int cols, float* const* dst, int D,
                        cudaStream_t stream);

}  // namespace gdn
