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
#include "gdn_host.h"
#include "gdn_norm.cuh"

namespace gdn {
namespace {

template <int TPR, int NV, int V, typename TX, typename T>
__global__ void __launch_bounds__(TPR ? kNormThreads : kNormMaxThreads)
    gated_norm_kernel(const GatedNormArgs a) {
  __shared__ float buf[2][1][16];
  int turn = 0;
  const int tpr = TPR ? TPR : blockDim.x, t = threadIdx.x % tpr;
  const int per = TPR ? kNormThreads / TPR : 1;
  float w[NV][V];
  load_weight<V, NV>(w, a.w, a.offset, 1.f, t, tpr, a.D);
  const float inv = 1.f / float(a.D);
  constexpr int kStages = stages(sizeof(TX) + sizeof(T));
  extern __shared__ __align__(16) unsigned char smem[];
  [[maybe_unused]] unsigned char* top = smem;
  [[maybe_unused]] const Ring<TX, V, NV, kStages> rx(top);
  [[maybe_unused]] const Ring<T, V, NV, kStages> rz(top);
  const long long stride = (long long)gridDim.x * per;
  const int sub = threadIdx.x / tpr;
  const auto fetch = [&](int stage, long long row) {
    if constexpr (kStaged<NV, V>) {
      if (row < a.rows + per) {  // (a whole CTA's rows past the end: nothing to copy)
        const int D = row < a.rows ? a.D : 0;
        const size_t at = size_t(row < a.rows ? row : 0) * a.D;
        rx.fetch(stage, static_cast<const TX*>(a.x) + at, t, tpr, D);
        if (a.z) rz.fetch(stage, static_cast<const T*>(a.z) + at, t, tpr, D);
      }
      copies_commit();
    }
  };
  const long long first = (long long)blockIdx.x * per;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i, first + i * stride + sub);
  int stage = 0;
  for (long long row0 = first; row0 < a.rows; row0 += stride) {
    const long long row = row0 + sub;
    const bool on = row < a.rows;
    const size_t at = size_t(on ? row : 0) * a.D;
    const int D = on ? a.D : 0;
    Vec<TX, V> x[NV];
    Vec<T, V> z[NV];
    if constexpr (kStaged<NV, V>) {
      copies_wait<kStages>();
      rx.take(x, stage);
      if (a.z) rz.take(z, stage);
      fetch(stage == 0 ? kStages - 1 : stage - 1, row + (kStages - 1) * stride);
      stage = stage == kStages - 1 ? 0 : stage + 1;
    } else {
      load_row<TX, V, NV>(x, static_cast<const TX*>(a.x) + at, t, tpr, D);
      if (a.z) load_row<T, V, NV>(z, static_cast<const T*>(a.z) + at, t, tpr, D);
    }
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) s[0] = fmaf(to_f(x[j].v[e]), to_f(x[j].v[e]), s[0]);
    row_sum<TPR, 1>(s, buf, turn);
    const float rstd = rsqrtf(fmaf(s[0], inv, a.eps));
    float y[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        y[j][e] = to_f(x[j].v[e]) * rstd * w[j][e];
        if (a.z) y[j][e] *= gate(a.act, to_f(z[j].v[e]));
      }
    store_row<T, V, NV>(static_cast<T*>(a.y) + at, y, t, tpr, D);
  }
}

template <int TPR, int NV, int V, typename TX, typename T>
__global__ void __launch_bounds__(TPR ? kNormThreads : kNormMaxThreads)
    gated_norm_backward_kernel(const GatedNormArgs a) {
  __shared__ float buf[2][2][16];
  __shared__ float groups[TPR ? kNormThreads * NV * V : 1];
  int turn = 0;
  const int tpr = TPR ? TPR : blockDim.x, t = threadIdx.x % tpr;
  const int per = TPR ? kNormThreads / TPR : 1;
  float w[NV][V], dw[NV][V];
  load_weight<V, NV>(w, a.w, a.offset, 1.f, t, tpr, a.D);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[j][e] = 0.f;
  const float inv = 1.f / float(a.D);
  constexpr int kStages = stages(sizeof(TX) + 2 * sizeof(T));
  extern __shared__ __align__(16) unsigned char smem[];
  [[maybe_unused]] unsigned char* top = smem;
  [[maybe_unused]] const Ring<TX, V, NV, kStages> rx(top);
  [[maybe_unused]] const Ring<T, V, NV, kStages> rd(top);
  [[maybe_unused]] const Ring<T, V, NV, kStages> rz(top);
  const long long stride = (long long)gridDim.x * per;
  const int sub = threadIdx.x / tpr;
  const auto fetch = [&](int stage, long long row) {
    if constexpr (kStaged<NV, V>) {
      if (row < a.rows + per) {  // (a whole CTA's rows past the end: nothing to copy)
        const int D = row < a.rows ? a.D : 0;
        const size_t at = size_t(row < a.rows ? row : 0) * a.D;
        rx.fetch(stage, static_cast<const TX*>(a.x) + at, t, tpr, D);
        rd.fetch(stage, static_cast<const T*>(a.dy) + at, t, tpr, D);
        if (a.z) rz.fetch(stage, static_cast<const T*>(a.z) + at, t, tpr, D);
      }
      copies_commit();
    }
  };
  const long long first = (long long)blockIdx.x * per;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i, first + i * stride + sub);
  int stage = 0;
  for (long long row0 = first; row0 < a.rows; row0 += stride) {
    const long long row = row0 + sub;
    const bool on = row < a.rows;
    const size_t at = size_t(on ? row : 0) * a.D;
    const int D = on ? a.D : 0;
    Vec<TX, V> x[NV];
    Vec<T, V> z[NV], dy[NV];
    if constexpr (kStaged<NV, V>) {
      copies_wait<kStages>();
      rx.take(x, stage);
      rd.take(dy, stage);
      if (a.z) rz.take(z, stage);
      fetch(stage == 0 ? kStages - 1 : stage - 1, row + (kStages - 1) * stride);
      stage = stage == kStages - 1 ? 0 : stage + 1;
    } else {
      load_row<TX, V, NV>(x, static_cast<const TX*>(a.x) + at, t, tpr, D);
      load_row<T, V, NV>(dy, static_cast<const T*>(a.dy) + at, t, tpr, D);
      if (a.z) load_row<T, V, NV>(z, static_cast<const T*>(a.z) + at, t, tpr, D);
    }
    float u[NV][V], dz[NV][V], s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float xe = to_f(x[j].v[e]), d = to_f(dy[j].v[e]);
        float av = 1.f, da = 0.f;
        if (a.z) gate_slope(a.act, to_f(z[j].v[e]), &av, &da);
        u[j][e] = d * av;            // times w below: dw wants it without
        dz[j][e] = d * w[j][e] * da * xe;
        s[0] = fmaf(xe, xe, s[0]);
        s[1] = fmaf(u[j][e] * w[j][e], xe, s[1]);
      }
    row_sum<TPR, 2>(s, buf, turn);
    const float rstd = rsqrtf(fmaf(s[0], inv, a.eps));
    const float c = s[1] * inv * rstd * rstd;  // mean(u xh) rstd
    float dx[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float xe = to_f(x[j].v[e]);
        dw[j][e] = fmaf(u[j][e], xe * rstd, dw[j][e]);
        dx[j][e] = rstd * fmaf(-c, xe, u[j][e] * w[j][e]);
        dz[j][e] *= rstd;
      }
    store_row<TX, V, NV>(static_cast<TX*>(a.dx) + at, dx, t, tpr, D);
    if (a.z) store_row<T, V, NV>(static_cast<T*>(a.dz) + at, dz, t, tpr, D);
  }
  if (a.part)
    store_partial<TPR, V, NV>(a.part + size_t(blockIdx.x) * a.D, dw, groups, t, tpr, a.D);
}

constexpr long long kForwardCtas = 8;  // per SM

template <typename TX, typename T>
struct Forward {
  const GatedNormArgs& a;
  int sms;
  cudaStream_t stream;
  template <int TPR, int NV, int V>
  int run() {
    const int threads = norm_threads<TPR, NV, V>(a.D), per = TPR ? kNormThreads / TPR : 1;
    const long long groups = (a.rows + per - 1) / per;
    const int grid = int(groups < kForwardCtas * sms ? groups : kForwardCtas * sms);
    constexpr size_t kBytes = sizeof(TX) + sizeof(T);  // staged of a channel
    constexpr size_t kThread = kStaged<NV, V> ? stages(kBytes) * NV * V * kBytes : 0;
    constexpr int kMost = TPR ? kNormThreads : kNormMaxThreads;
    if (!raise_smem<&gated_norm_kernel<TPR, NV, V, TX, T>>(kThread * kMost)) return GDN_ERR_LAUNCH;
    gated_norm_kernel<TPR, NV, V, TX, T><<<grid, threads, kThread * threads, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
  }
};

template <typename TX, typename T>
struct Backward {
  const GatedNormArgs& a;
  int sms;
  cudaStream_t stream;
  template <int TPR, int NV, int V>
  int run() {
    const int threads = norm_threads<TPR, NV, V>(a.D), per = TPR ? kNormThreads / TPR : 1;
    const long long groups = (a.rows + per - 1) / per;
    const int most = norm_max_parts(a.rows, a.D);
    const int grid = int(groups < most ? groups : most);
    constexpr size_t kBytes = sizeof(TX) + 2 * sizeof(T);  // staged of a channel
    constexpr size_t kThread = kStaged<NV, V> ? stages(kBytes) * NV * V * kBytes : 0;
    constexpr int kMost = TPR ? kNormThreads : kNormMaxThreads;
    if (!raise_smem<&gated_norm_backward_kernel<TPR, NV, V, TX, T>>(kThread * kMost)) return GDN_ERR_LAUNCH;
    gated_norm_backward_kernel<TPR, NV, V, TX, T><<<grid, threads, kThread * threads, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_LAUNCH;
    return launch_reduce_parts(a.part, grid, a.D, &a.dw, a.D, stream);
  }
};

bool wide_ok(const GatedNormArgs& a) {
  const void* p[] = {a.x, a.z, a.w, a.y, a.dy, a.dx, a.dz, a.part};
  uintptr_t all = 0;
  for (const void* q : p) all |= reinterpret_cast<uintptr_t>(q);
  return (all & 15) == 0;
}

template <template <typename, typename> class Run>
int dispatch(const GatedNormArgs& a, int x_dtype, int dtype, int sms, cudaStream_t stream) {
  using B = __nv_bfloat16;
  const bool wide = wide_ok(a);
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
