// RMS norm of a row times the gate: the post-step behind o of a recurrence (rows
// are heads), and a plain pre-norm without a gate.
//
//   y = a(z) w xh,   xh = x rstd,   rstd = (mean x^2 + eps)^-1/2
//   u = dy a(z) w;  dx = rstd (u - xh mean(u xh));  dz = dy w xh a'(z);
//   dw = sum over rows of dy a(z) xh
//
// One read of every input and one write of every output: HBM bounds both
// directions.  The backward pass finds rstd and mean(u xh) in one sum over the
// row (sum x^2 and sum u x), and keeps dw in registers while a CTA walks its
// rows; the CTAs' partial sums are added by a second launch in a fixed order.
//
// Measured (of the measured 6554 GB/s): 524288 x 128 in bf16 67 to 75 us (82 to
// 91%; half of a run's writes are the one before's, still in L2), its gradient
// over 131072 x 128 with x in fp32 45 us (79%), of which the first launch takes 34:
// its bytes at 107% of that rate, a part of the writes being left in L2.  What is
// left is the second launch and the gap before it.
#include "gdn_norm.cuh"

namespace gdn {
namespace {

template <typename L, typename TX, typename T>
__global__ void __launch_bounds__(L::TH) gated_norm_kernel(const GatedNormArgs a) {
  constexpr int kAll = sizeof(TX) + sizeof(T), kStages = stages<L>(kAll);
  constexpr int P = L::P, G = L::G, NV = L::NV;
  using RX = Ring<L, TX, 0, kAll>;
  using RZ = Ring<L, T, sizeof(TX), kAll>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ SumBuffer<L, 1> buf;
  const Place<L> at(a.D);
  const long long stride = (long long)gridDim.x * L::kRows;
  long long row = (long long)blockIdx.x * L::kRows + at.sub, next = row;
  int stage = 0, turn = 0, to = 0;
  // copies row `next` to stage `to` and steps both
  const auto fetch = [&] {
    if (next - at.sub < a.rows) {
      const bool on = next < a.rows;
      const size_t o = size_t(on ? next : 0) * a.D;
      RX::fetch(smem, to, static_cast<const TX*>(a.x) + o, at, on);
      if (a.z) RZ::fetch(smem, to, static_cast<const T*>(a.z) + o, at, on);
    }
    copies_commit();
    next += stride;
    to = to == kStages - 1 ? 0 : to + 1;
  };
  if constexpr (kStages > 0) {
    RX::clear(smem, at);
    RZ::clear(smem, at);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch();
  }
  sum_init(buf);
  F<P> w[NV][G];
#pragma unroll
  for (int j = 0; j < NV; ++j) load_weight<L>(w[j], a.w, a.offset, j, at);
  const float inv = 1.f / float(a.D);
  for (; row - at.sub < a.rows; row += stride) {
    const bool on = !L::kShort || row < a.rows;
    const size_t o = size_t(on ? row : 0) * a.D;
    const TX* px = static_cast<const TX*>(a.x) + o;
    const T* pz = static_cast<const T*>(a.z) + o;
    F<P> x[NV][G], z[NV][G];
    if constexpr (kStages > 0) copies_wait<kStages>();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      RX::take(x[j], smem, stage, px, j, at, on);
      if (a.z) RZ::take(z[j], smem, stage, pz, j, at, on);
    }
    if constexpr (kStages > 0) {
      stage = stage == kStages - 1 ? 0 : stage + 1;
      fetch();
    }
    F<P> sq = all<P>(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < G; ++i) sq = fma(x[j][i], x[j][i], sq);
    float s[1] = {total(sq)};
    row_sum<L, 1>(s, buf, turn);
    const F<P> rstd = all<P>(rsqrtf(fmaf(s[0], inv, a.eps)));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        x[j][i] = mul(mul(x[j][i], rstd), w[j][i]);
        if (a.z) x[j][i] = mul(x[j][i], gate(a.act, z[j][i]));
      }
      if (on) store_vector<L, T>(static_cast<T*>(a.y) + o, x[j], j, at);
    }
  }
}

template <typename L, typename TX, typename T>
__global__ void __launch_bounds__(L::TH, L::TH == 512 && L::NV * L::V == 8 ? 2 : 1)
    gated_norm_backward_kernel(const GatedNormArgs a) {
  constexpr int kAll = sizeof(TX) + 2 * sizeof(T), kStages = stages<L>(kAll);
  constexpr int P = L::P, G = L::G, NV = L::NV;
  using RX = Ring<L, TX, 0, kAll>;
  using RD = Ring<L, T, sizeof(TX), kAll>;
  using RZ = Ring<L, T, sizeof(TX) + sizeof(T), kAll>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ SumBuffer<L, 2> buf;
  __shared__ float groups[L::kShort ? L::kRows * L::kMost : 1];
  const Place<L> at(a.D);
  const long long stride = (long long)gridDim.x * L::kRows;
  long long row = (long long)blockIdx.x * L::kRows + at.sub, next = row;
  int stage = 0, turn = 0, to = 0;
  const auto fetch = [&] {
    if (next - at.sub < a.rows) {
      const bool on = next < a.rows;
      const size_t o = size_t(on ? next : 0) * a.D;
      RX::fetch(smem, to, static_cast<const TX*>(a.x) + o, at, on);
      RD::fetch(smem, to, static_cast<const T*>(a.dy) + o, at, on);
      if (a.z) RZ::fetch(smem, to, static_cast<const T*>(a.z) + o, at, on);
    }
    copies_commit();
    next += stride;
    to = to == kStages - 1 ? 0 : to + 1;
  };
  if constexpr (kStages > 0) {
    RX::clear(smem, at);
    RD::clear(smem, at);
    RZ::clear(smem, at);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch();
  }
  sum_init(buf);
  F<P> w[NV][G], dw[NV][G];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_weight<L>(w[j], a.w, a.offset, j, at);
#pragma unroll
    for (int i = 0; i < G; ++i) dw[j][i] = all<P>(0.f);
  }
  const float inv = 1.f / float(a.D);
  for (; row - at.sub < a.rows; row += stride) {
    const bool on = !L::kShort || row < a.rows;
    const size_t o = size_t(on ? row : 0) * a.D;
    const TX* px = static_cast<const TX*>(a.x) + o;
    const T *pd = static_cast<const T*>(a.dy) + o, *pz = static_cast<const T*>(a.z) + o;
    F<P> x[NV][G], dy[NV][G], z[NV][G];
    if constexpr (kStages > 0) {
      copies_wait<kStages>();
      // over the stage before this one: of long rows at once (8192 x 4096: 70 us
      // against 82), of short ones behind this one's reads (131072 x 128: 45.6
      // against 46.2)
      if (!L::kShort) fetch();
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      RX::take(x[j], smem, stage, px, j, at, on);
      RD::take(dy[j], smem, stage, pd, j, at, on);
      if (a.z) RZ::take(z[j], smem, stage, pz, j, at, on);
    }
    if constexpr (kStages > 0) {
      stage = stage == kStages - 1 ? 0 : stage + 1;
      if (L::kShort) fetch();
    }
    F<P> sq = all<P>(0.f), su = all<P>(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < G; ++i) {
        sq = fma(x[j][i], x[j][i], sq);
        if (a.z) {
          F<P> av, da;
          gate_slope(a.act, z[j][i], &av, &da);
          z[j][i] = mul(mul(mul(dy[j][i], w[j][i]), x[j][i]), da);  // dz, but for rstd
          dy[j][i] = mul(dy[j][i], av);                             // u without w
        }
        su = fma(mul(dy[j][i], w[j][i]), x[j][i], su);
      }
    float s[2] = {total(sq), total(su)};
    row_sum<L, 2>(s, buf, turn);
    const float r = rsqrtf(fmaf(s[0], inv, a.eps));
    const F<P> rstd = all<P>(r), c = all<P>(-(s[1] * inv * r * r));  // -mean(u xh) rstd
    if (on) {  // (with eps = 0 the root of a row that is not there is infinite)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
          dw[j][i] = fma(dy[j][i], mul(x[j][i], rstd), dw[j][i]);
          x[j][i] = mul(rstd, fma(c, x[j][i], mul(dy[j][i], w[j][i])));
          if (a.z) z[j][i] = mul(z[j][i], rstd);
        }
        store_vector<L, TX>(static_cast<TX*>(a.dx) + o, x[j], j, at);
        if (a.z) store_vector<L, T>(static_cast<T*>(a.dz) + o, z[j], j, at);
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  store_partial<L>(a.part + size_t(blockIdx.x) * a.D, dw, groups, at);
}

// Threads of all CTAs per SM; more than are resident where CTAs end early.
constexpr int kForwardThreads = 2048, kBackwardThreads = 1024;

template <typename TX, typename T>
struct Forward {
  const GatedNormArgs& a;
  int sms;
  cudaStream_t stream;
  template <typename L>
  int run() {
    const int threads = norm_threads<L>(a.D);
    const long long groups = (a.rows + L::kRows - 1) / L::kRows;
    const int grid =
        even_grid<L>(std::min<long long>(groups, kForwardThreads / threads * (long long)sms));
    constexpr int kBytes = sizeof(TX) + sizeof(T);
    constexpr size_t kThread = stages<L>(kBytes) * L::NV * L::V * kBytes;
    if (!raise_smem<&gated_norm_kernel<L, TX, T>>(kThread * L::TH)) return GDN_ERR_LAUNCH;
    gated_norm_kernel<L, TX, T><<<grid, threads, kThread * threads, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
  }
};

template <typename TX, typename T>
struct Backward {
  const GatedNormArgs& a;
  int sms;
  cudaStream_t stream;
  template <typename L>
  int run() {
    const int threads = norm_threads<L>(a.D);
    const long long groups = (a.rows + L::kRows - 1) / L::kRows;
    const int per_sm = std::max(1, (L::kShort ? 512 : kBackwardThreads) / threads);
    const int grid = even_grid<L>(std::min(
        {groups, (long long)norm_max_parts(a.rows, a.D), (long long)per_sm * sms}));
    constexpr int kBytes = sizeof(TX) + 2 * sizeof(T);
    constexpr size_t kThread = stages<L>(kBytes) * L::NV * L::V * kBytes;
    if (!raise_smem<&gated_norm_backward_kernel<L, TX, T>>(kThread * L::TH)) return GDN_ERR_LAUNCH;
    gated_norm_backward_kernel<L, TX, T><<<grid, threads, kThread * threads, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_LAUNCH;
    return launch_reduce_parts(a.part, grid, a.D, &a.dw, a.D, stream);
  }
};

// How many elements every array starts on a multiple of: 4, 2 or 1.
int width(const GatedNormArgs& a, int x_dtype, int dtype) {
  const uintptr_t ex = x_dtype == GDN_BF16 ? 2 : 4, e = dtype == GDN_BF16 ? 2 : 4;
  const auto ok = [&](uintptr_t n) {
    return aligned(a.x, n * ex) && aligned(a.dx, n * ex) && aligned(a.z, n * e) &&
           aligned(a.y, n * e) && aligned(a.dy, n * e) && aligned(a.dz, n * e) &&
           aligned(a.w, n * 4);
  };
  return ok(4) ? 4 : ok(2) ? 2 : 1;
}

template <template <typename, typename> class Run, int LONG>
int dispatch(const GatedNormArgs& a, int x_dtype, int dtype, int sms, cudaStream_t stream) {
  using B = __nv_bfloat16;
  const int n = width(a, x_dtype, dtype);
  if (x_dtype == GDN_BF16)
    return dtype == GDN_BF16 ? with_layout<LONG, false>(a.D, n, Run<B, B>{a, sms, stream})
                             : with_layout<LONG, false>(a.D, n, Run<B, float>{a, sms, stream});
  return dtype == GDN_BF16 ? with_layout<LONG, false>(a.D, n, Run<float, B>{a, sms, stream})
                           : with_layout<LONG, false>(a.D, n, Run<float, float>{a, sms, stream});
}

}  // namespace

int launch_gated_norm(const GatedNormArgs& a, int x_dtype, int dtype, int sms,
                      cudaStream_t stream) {
  return dispatch<Forward, 4>(a, x_dtype, dtype, sms, stream);
}

int launch_gated_norm_backward(const GatedNormArgs& a, int x_dtype, int dtype, int sms,
                               cudaStream_t stream) {
  return dispatch<Backward, 2>(a, x_dtype, dtype, sms, stream);
}

}  // namespace gdn
