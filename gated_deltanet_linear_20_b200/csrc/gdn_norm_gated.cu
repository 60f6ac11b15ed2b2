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
#include "gdn_norm.cuh"

namespace gdn {
namespace {

template <typename L, typename TX, typename T>
__global__ void __launch_bounds__(L::TH) gated_norm_kernel(const GatedNormArgs a) {
  constexpr int kAll = sizeof(TX) + sizeof(T), kStages = stages(kAll), P = L::P, N = L::N;
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
  if constexpr (L::kStaged) {
    RX::clear(smem, at);
    RZ::clear(smem, at);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch();
  }
  F<P> w[N];
  load_weight<L>(w, a.w, a.offset, at);
  const float inv = 1.f / float(a.D);
  for (; row - at.sub < a.rows; row += stride) {
    const bool on = !L::kShort || row < a.rows;
    const size_t o = size_t(on ? row : 0) * a.D;
    F<P> x[N], z[N];
    if constexpr (L::kStaged) {
      copies_wait<kStages>();
      RX::take(x, smem, stage);
      if (a.z) RZ::take(z, smem, stage);
      stage = stage == kStages - 1 ? 0 : stage + 1;
      fetch();
    } else {
      load_row<L, TX>(x, static_cast<const TX*>(a.x) + o, at, on);
      if (a.z) load_row<L, T>(z, static_cast<const T*>(a.z) + o, at, on);
    }
    F<P> sq = all<P>(0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) sq = fma(x[i], x[i], sq);
    float s[1] = {total(sq)};
    row_sum<L, 1>(s, buf, turn);
    const F<P> rstd = all<P>(rsqrtf(fmaf(s[0], inv, a.eps)));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = mul(mul(x[i], rstd), w[i]);
      if (a.z) x[i] = mul(x[i], gate(a.act, z[i]));
    }
    store_row<L, T>(static_cast<T*>(a.y) + o, x, at, on);
  }
}

template <typename L, typename TX, typename T>
__global__ void __launch_bounds__(L::TH) gated_norm_backward_kernel(const GatedNormArgs a) {
  constexpr int kAll = sizeof(TX) + 2 * sizeof(T), kStages = stages(kAll), P = L::P, N = L::N;
  using RX = Ring<L, TX, 0, kAll>;
  using RD = Ring<L, T, sizeof(TX), kAll>;
  using RZ = Ring<L, T, sizeof(TX) + sizeof(T), kAll>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ SumBuffer<L, 2> buf;
  __shared__ float groups[L::kShort ? L::TH * L::NV * L::V : 1];
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
  if constexpr (L::kStaged) {
    RX::clear(smem, at);
    RD::clear(smem, at);
    RZ::clear(smem, at);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch();
  }
  F<P> w[N], dw[N];
  load_weight<L>(w, a.w, a.offset, at);
#pragma unroll
  for (int i = 0; i < N; ++i) dw[i] = all<P>(0.f);
  const float inv = 1.f / float(a.D);
  for (; row - at.sub < a.rows; row += stride) {
    const bool on = !L::kShort || row < a.rows;
    const size_t o = size_t(on ? row : 0) * a.D;
    F<P> x[N], dy[N], z[N];
    if constexpr (L::kStaged) {
      copies_wait<kStages>();
      RX::take(x, smem, stage);
      RD::take(dy, smem, stage);
      if (a.z) RZ::take(z, smem, stage);
      stage = stage == kStages - 1 ? 0 : stage + 1;
      fetch();
    } else {
      load_row<L, TX>(x, static_cast<const TX*>(a.x) + o, at, on);
      load_row<L, T>(dy, static_cast<const T*>(a.dy) + o, at, on);
      if (a.z) load_row<L, T>(z, static_cast<const T*>(a.z) + o, at, on);
    }
    F<P> sq = all<P>(0.f), su = all<P>(0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      sq = fma(x[i], x[i], sq);
      if (a.z) {
        F<P> av, da;
        gate_slope(a.act, z[i], &av, &da);
        z[i] = mul(mul(mul(dy[i], w[i]), x[i]), da);  // dz, but for rstd
        dy[i] = mul(dy[i], av);                       // u without w
      }
      su = fma(mul(dy[i], w[i]), x[i], su);
    }
    float s[2] = {total(sq), total(su)};
    row_sum<L, 2>(s, buf, turn);
    const float r = rsqrtf(fmaf(s[0], inv, a.eps));
    const F<P> rstd = all<P>(r), c = all<P>(-(s[1] * inv * r * r));  // -mean(u xh) rstd
#pragma unroll
    for (int i = 0; i < N; ++i) {
      dw[i] = fma(dy[i], mul(x[i], rstd), dw[i]);
      x[i] = mul(rstd, fma(c, x[i], mul(dy[i], w[i])));
    }
    store_row<L, TX>(static_cast<TX*>(a.dx) + o, x, at, on);
    if (a.z) {
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = mul(z[i], rstd);
      store_row<L, T>(static_cast<T*>(a.dz) + o, z, at, on);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  store_partial<L>(a.part + size_t(blockIdx.x) * a.D, dw, groups, at);
}

constexpr long long kForwardCtas = 16;  // per SM: 8 rows of a CTA at a time are resident

template <typename TX, typename T>
struct Forward {
  const GatedNormArgs& a;
  int sms;
  cudaStream_t stream;
  template <typename L>
  int run() {
    const long long groups = (a.rows + L::kRows - 1) / L::kRows;
    const int grid = int(std::min(groups, kForwardCtas * sms));
    constexpr size_t smem = ring_bytes<L>(sizeof(TX) + sizeof(T));
    if (!raise_smem<&gated_norm_kernel<L, TX, T>>(smem)) return GDN_ERR_LAUNCH;
    gated_norm_kernel<L, TX, T><<<grid, L::TH, smem, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
  }
  int run4096() { return run<Layout<256, 256, 4, 4>>(); }
};

template <typename TX, typename T>
struct Backward {
  const GatedNormArgs& a;
  int sms;
  cudaStream_t stream;
  template <typename L>
  int run() {
    const long long groups = (a.rows + L::kRows - 1) / L::kRows;
    const int grid = int(std::min<long long>(groups, norm_max_parts(a.rows, a.D)));
    constexpr size_t smem = ring_bytes<L>(sizeof(TX) + 2 * sizeof(T));
    if (!raise_smem<&gated_norm_backward_kernel<L, TX, T>>(smem)) return GDN_ERR_LAUNCH;
    gated_norm_backward_kernel<L, TX, T><<<grid, L::TH, smem, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_LAUNCH;
    return launch_reduce_parts(a.part, grid, a.D, &a.dw, a.D, stream);
  }
  int run4096() { return run<Layout<512, 512, 2, 4>>(); }
};

// Whether every array starts on four elements.
bool wide_ok(const GatedNormArgs& a, int x_dtype, int dtype) {
  const uintptr_t ex = x_dtype == GDN_BF16 ? 8 : 16, e = dtype == GDN_BF16 ? 8 : 16;
  return aligned(a.x, ex) && aligned(a.dx, ex) && aligned(a.z, e) && aligned(a.y, e) &&
         aligned(a.dy, e) && aligned(a.dz, e) && aligned(a.w, 16);
}

template <template <typename, typename> class Run>
int dispatch(const GatedNormArgs& a, int x_dtype, int dtype, int sms, cudaStream_t stream) {
  using B = __nv_bfloat16;
  const bool wide = wide_ok(a, x_dtype, dtype);
  if (x_dtype == GDN_BF16)
    return dtype == GDN_BF16 ? with_layout(a.D, wide, Run<B, B>{a, sms, stream})
                             : with_layout(a.D, wide, Run<B, float>{a, sms, stream});
  return dtype == GDN_BF16 ? with_layout(a.D, wide, Run<float, B>{a, sms, stream})
                           : with_layout(a.D, wide, Run<float, float>{a, sms, stream});
}

}  // namespace

int launch_gated_norm(const GatedNormArgs& a, int x_dtype, int dtype, int sms,
                      cudaStream_t stream) {
  return dispatch<Forward>(a, x_dtype, dtype, sms, stream);
}

int launch_gated_norm_backward(const GatedNormArgs& a, int x_dtype, int dtype, int sms,
                               cudaStream_t stream) {
  return dispatch<Backward>(a, x_dtype, dtype, sms, stream);
}

}  // namespace gdn
