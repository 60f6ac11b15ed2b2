// What the norm kernels share: the layout of a row over threads, its sums, the
// gate, and the copies of the next rows.
//
// A row of D channels is held by a group of threads, NV vectors of V channels
// each, so it is read from memory once, whatever is summed over it.  Short rows
// share a CTA, TPR = 8, 16 or 32 threads a row (vector j of thread t: channels
// (j TPR + t) V ..), and sum by shuffles; longer ones have a CTA of as many warps
// as they need (TPR 0), each with 32 NV V neighbouring channels.
//
// CTAs are persistent, and each thread copies its part of the next rows to shared
// memory asynchronously (a ring of two or three stages) while it works on the
// present one: the sums over a row and their barriers would leave the memory
// idle otherwise.  A thread reads only what it copied, so the ring needs no
// barrier.  (One bulk copy an array and row, by one thread, was slower: 524288 x
// 128 82 us against 67, 8192 x 4096 48 against 47.)  What is left is the
// instruction count, so that channels are worked on in pairs.
#pragma once

#include <algorithm>

#include "gdn_host.h"
#include "gdn_internal.h"
#include "gdn_vec.cuh"

namespace gdn {

// TH: threads of a CTA, the most of them where TPR is 0.
template <int TPR_, int TH_, int NV_, int V_, bool ODD = false>
struct Layout {
  static constexpr int TPR = TPR_, TH = TH_, NV = NV_, V = V_;
  static constexpr bool kShort = TPR > 0;               // several rows a CTA
  static constexpr bool kOdd = ODD;                     // rows of an odd number of channels
  static constexpr int kRows = kShort ? TH / (TPR > 0 ? TPR : 1) : 1;
  static constexpr int P = V >= 2 ? 2 : 1;              // channels worked on together
  static constexpr int G = V / P;                       // such groups of a vector
  static constexpr int kStep = (kShort ? TPR : 32) * V; // channels from vector to vector
  static constexpr int kMost = (kShort ? TPR : TH) * NV * V;  // channels
};

// Stages of a ring whose arrays have `bytes` a channel in all: three, or two, or
// none where the longest row leaves no room (or for single channels, which may
// have 2 bytes: copies have 4 at least).
template <typename L>
constexpr int stages(size_t bytes) {
  const size_t fit = 220 * 1024 / (bytes * L::TH * L::NV * L::V);
  return L::V == 1 || fit < 2 ? 0 : fit < 3 ? 2 : 3;
}
// Threads of a CTA for rows of D channels.
template <typename L>
int norm_threads(int D) {
  const int most = D + (L::kOdd ? 1 : 0);  // with the shift of an odd row
  return L::kShort ? L::TH : (most + L::NV * L::V * 32 - 1) / (L::NV * L::V * 32) * 32;
}

// This thread's place: its row among the CTA's, the first channel of its vectors.
// Of rows with an odd number of channels every second starts in the middle of an
// aligned pair: there the pairs are shifted, -1 and 0 being the first.  A thread
// stays with rows of one kind (CTAs step by an even number of rows).
template <typename L>
struct Place {
  int sub, c0, D;
  __device__ __forceinline__ explicit Place(int d)
      : sub(L::kShort ? threadIdx.x / (L::kShort ? L::TPR : 1) : 0),
        c0(L::kShort ? threadIdx.x % (L::kShort ? L::TPR : 1) * L::V
                     : (threadIdx.x >> 5) * (L::NV * L::kStep) + (threadIdx.x & 31) * L::V),
        D(d) {
    if (L::kOdd) c0 -= (blockIdx.x * L::kRows + sub) & 1;
  }
  __device__ __forceinline__ int channel(int j) const { return c0 + j * L::kStep; }
  __device__ __forceinline__ bool has(int j) const { return channel(j) < D; }
  // channel e of vector j is one of the row's; all of them are
  __device__ __forceinline__ bool in(int j, int e) const {
    return !L::kOdd ? has(j) : channel(j) + e < D && (e > 0 || channel(j) >= 0);
  }
  __device__ __forceinline__ bool whole(int j) const {
    return in(j, 0) && in(j, L::V - 1);
  }
};
// Rows that the CTAs of a launch step by are even in number.
template <typename L>
int even_grid(long long grid) {
  return int(L::kOdd && L::kRows == 1 && grid > 1 ? grid & ~1LL : grid);
}

// The channels of a vector, in groups.
template <typename L, typename T>
__device__ __forceinline__ void spread(F<L::P> (&r)[L::G], const Vec<T, L::V>& x) {
#pragma unroll
  for (int e = 0; e < L::V; ++e) r[e / L::P].v[e % L::P] = to_f(x.v[e]);
}
// Vector j of a row at p, channels that are not the row's as zeros.
template <typename L, typename T>
__device__ __forceinline__ void load_vector(F<L::P> (&r)[L::G], const T* p, int j,
                                            const Place<L>& at) {
  Vec<T, L::V> x{};
  if (!L::kOdd) {
    if (at.has(j)) x = load<T, L::V>(p + at.channel(j));
  } else {
#pragma unroll
    for (int e = 0; e < L::V; ++e)
      if (at.in(j, e)) x.v[e] = p[at.channel(j) + e];
  }
  spread<L, T>(r, x);
}
template <typename L, typename T>
__device__ __forceinline__ void store_vector(T* p, const F<L::P> (&r)[L::G], int j,
                                             const Place<L>& at) {
  float x[L::V];
#pragma unroll
  for (int e = 0; e < L::V; ++e) x[e] = r[e / L::P].v[e % L::P];
  if (at.whole(j)) {
    store<T, L::V>(p + at.channel(j), x);
  } else if (L::kOdd) {
#pragma unroll
    for (int e = 0; e < L::V; ++e)
      if (at.in(j, e)) p[at.channel(j) + e] = from_f<T>(x[e]);
  }
}

// One input array in the ring: BEFORE bytes a channel of other arrays lie before
// it in a stage of ALL bytes a channel.
template <typename L, typename T, int BEFORE, int ALL, int STAGES = stages<L>(ALL)>
struct Ring {
  using E = Vec<T, L::V>;
  static constexpr int kStages = STAGES;
  __device__ __forceinline__ static E* slot(unsigned char* smem, int stage, int j) {
    const unsigned threads = L::kShort ? L::TH : blockDim.x;
    E* p = reinterpret_cast<E*>(smem + (stage * ALL + BEFORE) * (threads * L::NV * L::V));
    return L::kShort ? p + j * L::TH + threadIdx.x
                     : p + ((threadIdx.x >> 5) * L::NV + j) * 32 + (threadIdx.x & 31);
  }
  // Channels past D stay zero in every stage.
  __device__ __forceinline__ static void clear(unsigned char* smem, const Place<L>& at) {
#pragma unroll
    for (int s = 0; s < kStages; ++s)
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
        // (an aligned address also where nothing is read: p is row 0 then)
        const E* src =
            reinterpret_cast<const E*>(L::kOdd && L::kShort && !on ? p : p + at.channel(j));
        // a pair past the row's end has one channel, the other is zero
        const int bytes = L::kOdd && !at.in(j, L::V - 1) ? int(sizeof(T)) : int(sizeof(E));
        if (L::kShort || L::kOdd)
          copy_async(slot(smem, stage, j), src, on ? bytes : 0);
        else
          copy_async(slot(smem, stage, j), src);
      }
  }
  // Vector j of the present row: from the ring, or (no stages) from memory.
  __device__ __forceinline__ static void take(F<L::P> (&r)[L::G], unsigned char* smem, int stage,
                                              const T* p, int j, const Place<L>& at, bool on) {
    if constexpr (kStages > 0) {
      spread<L, T>(r, *slot(smem, stage, j));
      if (L::kOdd && at.channel(j) < 0) r[0].v[0] = 0.f;  // the row's before
    } else if (on) {
      load_vector<L, T>(r, p, j, at);
    } else {
      spread<L, T>(r, E{});
    }
  }
};

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int STAGES>
__device__ __forceinline__ void copies_wait() {  // for the oldest stage in flight
  asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
}

// The weights of vector j, `offset` added; ones without any.  (Channels that are
// not the row's have inputs of zero, whatever their weight.)
template <typename L>
__device__ __forceinline__ void load_weight(F<L::P> (&w)[L::G], const float* p, float offset, int j,
                                            const Place<L>& at) {
#pragma unroll
  for (int i = 0; i < L::G; ++i) w[i] = all<L::P>(p ? 0.f : 1.f);
  if (p && at.has(j)) {
    load_vector<L, float>(w, p, j, at);
#pragma unroll
    for (int i = 0; i < L::G; ++i) w[i] = add(w[i], all<L::P>(offset));
  }
}

template <int P>
__device__ __forceinline__ float total(F<P> a) {
  return P == 2 ? a.v[0] + a.v[P - 1] : a.v[0];
}

// Sums of K values over the threads of a row; every thread gets them.  For rows
// of a CTA `buf` holds two sets, used in turn, so that one barrier a sum is
// enough.  The order of the additions is fixed.
template <typename L, int K>
struct SumBuffer {
  float part[2][K == 1 ? 1 : 4][16];
};
// Before the first sum (the places of warps that there are not stay zero).
template <typename L, int K>
__device__ __forceinline__ void sum_init(SumBuffer<L, K>& buf) {
  if constexpr (!L::kShort) {
    for (int i = threadIdx.x; i < 2 * (K == 1 ? 1 : 4) * 16; i += blockDim.x)
      (&buf.part[0][0][0])[i] = 0.f;
    __syncthreads();
  }
}
template <typename L, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], SumBuffer<L, K>& buf, int& turn) {
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
      v[0] = buf.part[turn][0][lane & 15];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) v[0] = halve(v[0], o);
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
    x = buf.part[turn][mine][lane & 7] + buf.part[turn][mine][(lane & 7) + 8];
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) x = halve(x, o);
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, x, 8 * k);
    turn ^= 1;
  }
}

// exp(z) and 1 / z by the approximate instructions: two units in the last place and |z|
// half steps for the product in the exponent; one unit.  Results below the normal
// numbers are zero, so that a gate below -87.3 is (its value is less than 1e-36; with
// such results kept 524288 x 128 took 74 us against 69, its gradient 122 against 117).
__device__ __forceinline__ float power(float z) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * 1.4426950408889634f));
  return e;
}
__device__ __forceinline__ float inverse(float z) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(z));
  return r;
}
// The gate's value, with p = 1 / (1 + exp(-z)): p z or p.  An overflowing exponential
// gives 0.
template <int P>
__device__ __forceinline__ F<P> gate(int act, F<P> z) {
  F<P> p;
#pragma unroll
  for (int e = 0; e < P; ++e) {
    p.v[e] = inverse(1.f + power(-z.v[e]));
    z.v[e] = act == GDN_GATE_SILU ? z.v[e] : 1.f;
  }
  return mul(z, p);
}
// Its value and slope, with q = 1 - p = 1 / (1 + exp(z)): p (1 + z q), or p q.  With e =
// exp(-|z|) the larger of p and q is 1 / (1 + e), the smaller e times that: as a
// difference q would lose its bits where p is close to one.
template <int P>
__device__ __forceinline__ void gate_slope(int act, F<P> z, F<P>* a, F<P>* da) {
  F<P> p, q;
#pragma unroll
  for (int e = 0; e < P; ++e) {
    const float x = power(-fabsf(z.v[e])), r = inverse(1.f + x), s = x * r;
    p.v[e] = z.v[e] < 0.f ? s : r;
    q.v[e] = z.v[e] < 0.f ? r : s;
    z.v[e] = act == GDN_GATE_SILU ? z.v[e] : 1.f;
  }
  *a = mul(z, p);
  *da = mul(p, fma(z, q, all<P>(act == GDN_GATE_SILU ? 1.f : 0.f)));
}

// A CTA's partial sums of one weight gradient, one row of D values: its rows'
// groups of threads are added in order through shared memory.
template <typename L>
__device__ __forceinline__ void store_partial(float* part, const F<L::P> (&acc)[L::NV][L::G],
                                              float* smem, const Place<L>& at) {
  if constexpr (!L::kShort) {
#pragma unroll
    for (int j = 0; j < L::NV; ++j)
#pragma unroll
      for (int e = 0; e < L::V; ++e)
        if (at.in(j, e)) part[at.channel(j) + e] = acc[j][e / L::P].v[e % L::P];
  } else {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < L::NV; ++j)
#pragma unroll
      for (int e = 0; e < L::V; ++e)
        if (at.in(j, e))
          smem[at.sub * L::kMost + at.channel(j) + e] = acc[j][e / L::P].v[e % L::P];
    __syncthreads();
    for (int c = threadIdx.x; c < at.D; c += L::TH) {
      float s = 0.f;
      for (int i = 0; i < L::kRows; ++i) s += smem[i * L::kMost + c];
      part[c] = s;
    }
  }
}

// Calls f.template run<Layout>() with the layout for rows of D channels: vectors
// of four where D is a multiple of 4 and every array starts on one (`width` 4: 8
// bytes of bf16, 16 of fp32), pairs where they start on one, else single channels.
// Pairs and single channels have layouts of 16 channels a thread before those of 32,
// whose sums leave the registers (gradients of the residual norm, 2000 x 4097 in bf16:
// 111 us against 552).
// LONG: vectors of a thread in rows of 257 to 4096 channels.  TRIM: rows of up to
// 6144 channels in a layout of their own, whose smaller stages leave room in shared
// memory (the residual norm's gradients, 2730 x 6144 in bf16: 64 us against 78; its
// forward pass 36 against 31, so without it).
template <int LONG, bool TRIM, typename F>
int with_layout(int D, int width, F&& f) {
  if (width == 4 && D % 4 == 0) {
    if (D <= 64) return f.template run<Layout<8, 256, 2, 4>>();
    if (D <= 128) return f.template run<Layout<16, 256, 2, 4>>();
    if (D <= 256) return f.template run<Layout<32, 256, 2, 4>>();
    if (D <= 4096) return f.template run<Layout<0, 1024 / LONG, LONG, 4>>();
    if constexpr (TRIM)
      if (D <= 6144) return f.template run<Layout<0, 384, 4, 4>>();
    if (D <= 8192) return f.template run<Layout<0, 512, 4, 4>>();
    return f.template run<Layout<0, 512, 8, 4>>();
  }
  if (width >= 2 && D % 2 == 0) {
    if (D <= 32) return f.template run<Layout<8, 256, 2, 2>>();
    if (D <= 64) return f.template run<Layout<16, 256, 2, 2>>();
    if (D <= 256) return f.template run<Layout<32, 256, 4, 2>>();
    if (D <= 4096) return f.template run<Layout<0, 512, 4, 2>>();
    if (D <= 8192) return f.template run<Layout<0, 512, 8, 2>>();
    return f.template run<Layout<0, 512, 16, 2>>();
  }
  if (width >= 2) {
    if (D < 32) return f.template run<Layout<8, 256, 2, 2, true>>();
    if (D < 64) return f.template run<Layout<16, 256, 2, 2, true>>();
    if (D < 256) return f.template run<Layout<32, 256, 4, 2, true>>();
    if (D < 4096) return f.template run<Layout<0, 512, 4, 2, true>>();
    if (D < 8192) return f.template run<Layout<0, 512, 8, 2, true>>();
    return f.template run<Layout<0, 512, 17, 2, true>>();
  }
  if (D <= 256) return f.template run<Layout<32, 256, 8, 1>>();
  if (D <= 4096) return f.template run<Layout<0, 512, 8, 1>>();
  if (D <= 8192) return f.template run<Layout<0, 512, 16, 1>>();
  return f.template run<Layout<0, 512, 32, 1>>();
}

// dst[i] = sum over parts p < n of part[p][i], i < cols.
int launch_reduce_parts(const float* part, int n, int cols, float* const* dst, int D,
                        cudaStream_t stream);

}  // namespace gdn
