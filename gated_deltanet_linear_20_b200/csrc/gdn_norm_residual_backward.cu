// The gradients of the step between two blocks (gdn_norm_residual.cuh).
//
// Measured (of the measured 6554 GB/s): 4096 x 4096 with everything on and r in fp32
// 75 us (75%), 8192 x 4096 in bf16 without a gate 103 us (60%).  They are bound by
// their instructions (70 a channel; a warp issues in half the cycles) and by
// registers: 24 sums, 24 weights and five inputs of 8 channels a thread leave one CTA
// of 512 threads an SM.
#include "gdn_norm_residual.cuh"

namespace gdn {
namespace {

// A thread with more than 8 channels has no registers for its inputs and weights
// beside the sums: for every pass over the row it takes each vector again from the
// ring (or from memory) and the weights from shared memory, as many of the three as
// fit behind a ring of two stages, the others from the cache.  In fours only: pairs
// have no ring and took longer with less of the L1 cache.  (2730 x 6144 and 2048 x
// 8192 in bf16 64 and 87 us against 93 and 92 with all weights from the cache.  Held
// to 128 registers although 384 threads may have 168: 64 against 70, and 101 with
// three stages besides.)
template <typename L>
constexpr bool keeps() {
  return L::NV * L::V <= 8;
}
template <typename L>
constexpr int backward_stages(size_t bytes) {
  return keeps<L>() ? stages<L>(bytes) : std::min(2, stages<L>(bytes));
}
template <typename L>
constexpr int shared_weights(size_t ring) {  // ring: its bytes a channel
  return keeps<L>() || L::V < 4 ? 0 : std::min<int>(3, (224 * 1024 - ring * L::kMost) / (4 * L::kMost));
}
template <typename L, typename T, typename TR>
__global__ void __launch_bounds__(keeps<L>() ? L::TH : 512)  // 128 registers also for fewer threads
    residual_norm_backward_kernel(const ResidualNormArgs a) {
  constexpr int kT = sizeof(T), kR = sizeof(TR), kAll = 3 * kT + 2 * kR;
  constexpr int kStages = backward_stages<L>(kAll);
  constexpr int P = L::P, G = L::G, NV = L::NV;
  constexpr bool kKeep = keeps<L>();
  constexpr int kShared = shared_weights<L>(kStages * kAll);
  constexpr int KV = kKeep ? NV : 1;  // vectors kept
  using RR = Ring<L, TR, 0, kAll, kStages>;
  using RG = Ring<L, TR, kR, kAll, kStages>;
  using RD = Ring<L, T, 2 * kR, kAll, kStages>;
  using RX = Ring<L, T, 2 * kR + kT, kAll, kStages>;
  using RZ = Ring<L, T, 2 * kR + 2 * kT, kAll, kStages>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ SumBuffer<L, 3> buf3;
  __shared__ SumBuffer<L, 1> buf1;
  __shared__ float groups[L::kShort ? L::kRows * L::kMost : 1];
  const Place<L> at(a.D);
  const long long stride = (long long)gridDim.x * L::kRows;
  long long row = (long long)blockIdx.x * L::kRows + at.sub, next = row;
  int stage = 0, turn3 = 0, turn1 = 0, to = 0;
  const auto fetch = [&] {
    if (next - at.sub < a.rows) {
      const bool on = next < a.rows;
      const size_t o = size_t(on ? next : 0) * a.D;
      RR::fetch(smem, to, static_cast<const TR*>(a.r) + o, at, on);
      RD::fetch(smem, to, static_cast<const T*>(a.dy) + o, at, on);
      RX::fetch(smem, to, static_cast<const T*>(a.x) + o, at, on);
      if (a.dr_out) RG::fetch(smem, to, static_cast<const TR*>(a.dr_out) + o, at, on);
      if (a.z) RZ::fetch(smem, to, static_cast<const T*>(a.z) + o, at, on);
    }
    copies_commit();
    next += stride;
    to = to == kStages - 1 ? 0 : to + 1;
  };
  if constexpr (kStages > 0) {
    RR::clear(smem, at);
    RG::clear(smem, at);
    RD::clear(smem, at);
    RX::clear(smem, at);
    RZ::clear(smem, at);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch();
  }
  sum_init(buf3);
  sum_init(buf1);
  F<P> w[KV][G], wp[KV][G], sc[KV][G], dw[NV][G], dwp[NV][G], dsc[NV][G];
  // Weight n (w, w_post, scale) of vector j: from memory; its place in shared memory,
  // which only this thread reads; from there, if it is one of those kept there.
  const auto load_one = [&](F<P>(&to)[G], int n, int j) {
    load_weight<L>(to, n == 0 ? a.w : n == 1 ? a.w_post : a.scale, n < 2 ? a.offset : 0.f, j, at);
  };
  const auto place = [&](int n, int j) {
    auto* first = reinterpret_cast<Vec<float, L::V>*>(
        smem + size_t(blockDim.x) * (NV * L::V) * (kStages * kAll + 4 * n));
    return first + ((threadIdx.x >> 5) * NV + j) * 32 + (threadIdx.x & 31);
  };
  const auto weight = [&](F<P>(&to)[G], int n, int j) {
    if (n < kShared)
      spread<L, float>(to, *place(n, j));
    else
      load_one(to, n, j);
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (kKeep) {
      load_one(w[j], 0, j);
      load_one(wp[j], 1, j);
      load_one(sc[j], 2, j);
    }
#pragma unroll
    for (int n = 0; n < kShared; ++n) {
      F<P> x[G];
      load_one(x, n, j);
#pragma unroll
      for (int e = 0; e < L::V; ++e) place(n, j)->v[e] = x[e / P].v[e % P];
    }
#pragma unroll
    for (int i = 0; i < G; ++i) dw[j][i] = dwp[j][i] = dsc[j][i] = all<P>(0.f);
  }
  const float inv = 1.f / float(a.D);
  for (; row - at.sub < a.rows; row += stride) {
    const bool on = !L::kShort || row < a.rows;
    const size_t o = size_t(on ? row : 0) * a.D;
    const T *px = static_cast<const T*>(a.x) + o, *pz = static_cast<const T*>(a.z) + o,
            *pd = static_cast<const T*>(a.dy) + o;
    const TR *pr = static_cast<const TR*>(a.r) + o, *pg = static_cast<const TR*>(a.dr_out) + o;
    F<P> x[KV][G], z[KV][G], dy[KV][G], r[KV][G], q[KV][G], v[NV][G];
    if constexpr (kStages > 0) {
      copies_wait<kStages>();
      if (!kKeep) fetch();  // over the stage before this one
    }
    const int here = stage;
    // the vectors of the first sum, and those of the second besides
    const auto take = [&](int j, bool rest) {
      const int k = kKeep ? j : 0;
      if (!kKeep || !rest) {
        RR::take(r[k], smem, here, pr, j, at, on);
        RD::take(dy[k], smem, here, pd, j, at, on);
        RX::take(x[k], smem, here, px, j, at, on);
      }
      if (kKeep != rest) {
        if (a.dr_out) {
          RG::take(q[k], smem, here, pg, j, at, on);
        } else {
#pragma unroll
          for (int i = 0; i < G; ++i) q[k][i] = all<P>(0.f);
        }
        if (a.z) RZ::take(z[k], smem, here, pz, j, at, on);
      }
    };
    F<P> s0 = all<P>(0.f), s1 = s0, s2 = s0;
    if (kKeep) {
#pragma unroll
      for (int j = 0; j < NV; ++j) take(j, false);
      if constexpr (kStages > 0) fetch();
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = kKeep ? j : 0;
      if (!kKeep) {
        take(j, false);
        weight(w[k], 0, j);
      }
#pragma unroll
      for (int i = 0; i < G; ++i) {
        s0 = fma(r[k][i], r[k][i], s0);
        s1 = fma(mul(dy[k][i], w[k][i]), r[k][i], s1);
        s2 = fma(x[k][i], x[k][i], s2);
      }
    }
    float s[3] = {total(s0), total(s1), total(s2)};
    row_sum<L, 3>(s, buf3, turn3);
    const float rs = rsqrtf(fmaf(s[0], inv, a.eps));
    const float rx = a.w_post ? rsqrtf(fmaf(s[2], inv, a.eps)) : 1.f;
    const F<P> rr = all<P>(rs), c = all<P>(-(s[1] * inv * rs * rs)), rp = all<P>(rx);
    F<P> sm = all<P>(0.f);
    if (on) {  // (with eps = 0 the roots of a row that is not there are infinite)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int k = kKeep ? j : 0;
        if (!kKeep) {
          take(j, true);
          weight(w[k], 0, j);
          weight(wp[k], 1, j);
          weight(sc[k], 2, j);
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
          q[k][i] = fma(rr, fma(c, r[k][i], mul(dy[k][i], w[k][i])), q[k][i]);
          dw[j][i] = fma(dy[k][i], mul(r[k][i], rr), dw[j][i]);
          x[k][i] = mul(x[k][i], rp);  // xh
          const F<P> u = mul(x[k][i], wp[k][i]);
          F<P> qa = q[k][i];
          if (a.z) {
            F<P> av, da;
            gate_slope(a.act, z[k][i], &av, &da);
            qa = mul(qa, av);
            z[k][i] = mul(mul(mul(q[k][i], sc[k][i]), u), da);  // dz
          }
          dsc[j][i] = fma(qa, u, dsc[j][i]);
          v[j][i] = mul(qa, sc[k][i]);
          dwp[j][i] = fma(v[j][i], x[k][i], dwp[j][i]);
          sm = fma(v[j][i], u, sm);
        }
        store_vector<L, TR>(static_cast<TR*>(a.dr) + o, q[k], j, at);
        if (a.z) store_vector<L, T>(static_cast<T*>(a.dz) + o, z[k], j, at);
      }
    }
    float mean = 0.f;  // of v w_post xh
    if (a.w_post) {
      float m[1] = {total(sm)};
      row_sum<L, 1>(m, buf1, turn1);
      mean = m[0] * inv;
    }
    if (on) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (a.w_post) {
          const int k = kKeep ? j : 0;
          if (!kKeep) {
            RX::take(x[k], smem, here, px, j, at, on);
            weight(wp[k], 1, j);
#pragma unroll
            for (int i = 0; i < G; ++i) x[k][i] = mul(x[k][i], rp);
          }
#pragma unroll
          for (int i = 0; i < G; ++i)
            v[j][i] = mul(rp, fma(all<P>(-mean), x[k][i], mul(v[j][i], wp[k][i])));
        }
        store_vector<L, T>(static_cast<T*>(a.dx) + o, v[j], j, at);
      }
    }
    if constexpr (kStages > 0) stage = stage == kStages - 1 ? 0 : stage + 1;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // partial gradients of the weights that there are: w, then w_post, then scale
  float* part = a.part + size_t(blockIdx.x) * a.D * a.weights;
  store_partial<L>(part, dw, groups, at);
  if (a.w_post) store_partial<L>(part += a.D, dwp, groups, at);
  if (a.scale) store_partial<L>(part += a.D, dsc, groups, at);
}

// Threads of all CTAs per SM.
constexpr int kThreads = 512;

template <typename T, typename TR>
struct Backward {
  const ResidualNormArgs& a;
  int sms;
  cudaStream_t stream;
  template <typename L>
  int run() {
    const int threads = norm_threads<L>(a.D);
    const long long groups = (a.rows + L::kRows - 1) / L::kRows;
    const int per_sm = std::max(1, kThreads / threads);
    const int grid = even_grid<L>(std::min(
        {groups, (long long)norm_max_parts(a.rows, a.D), (long long)per_sm * sms}));
    constexpr int kBytes = 3 * sizeof(T) + 2 * sizeof(TR);
    constexpr int kRing = backward_stages<L>(kBytes) * kBytes;
    constexpr size_t kThread = L::NV * L::V * size_t(kRing + 4 * shared_weights<L>(kRing));
    if (!raise_smem<&residual_norm_backward_kernel<L, T, TR>>(kThread * L::TH))
      return GDN_ERR_LAUNCH;
    residual_norm_backward_kernel<L, T, TR><<<grid, threads, kThread * threads, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_LAUNCH;
    float* dst[3] = {a.dw, a.w_post ? a.dw_post : a.dscale, a.dscale};
    return launch_reduce_parts(a.part, grid, a.D * a.weights, dst, a.D, stream);
  }
};

}  // namespace

int launch_residual_norm_backward(const ResidualNormArgs& a, int dtype, int r_dtype, int sms,
                                  cudaStream_t stream) {
  return dispatch<Backward, 2, true>(a, dtype, r_dtype, sms, stream);
}

}  // namespace gdn
