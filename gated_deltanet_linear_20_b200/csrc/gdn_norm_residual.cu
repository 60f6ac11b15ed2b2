// The step between two blocks: norm behind the block, its gate and scale, the
// residual sum and the norm before the next block, in one pass.
//
//   u  = w_post x rstd_x  (or x);   r' = r + scale a(z) u;   y = w r' rstd_r
// backward, at the kept sum r' (rh = r' rstd_r, xh = x rstd_x):
//   dr = dr' + rstd_r (dy w - rh mean(dy w rh));   dw = sum dy rh
//   dscale = sum dr a u;   dz = dr scale u a';   v = dr scale a
//   dx = rstd_x (v w_post - xh mean(v w_post xh))  (or v);   dw_post = sum v xh
//
// HBM bounds both directions.  A row stays in registers through both norms: the
// forward pass sums it twice, the backward pass twice as well (all that needs
// only inputs in the first sum).  y comes from the fp32 sum before r' is rounded
// to its type.  The weight gradients of a CTA's rows stay in registers and the
// CTAs' partial sums are added by a second launch in a fixed order.
#include "gdn_host.h"
#include "gdn_norm.cuh"

namespace gdn {
namespace {

template <int TPR, int NV, int V, typename T, typename TR>
__global__ void __launch_bounds__(TPR ? kNormThreads : kNormMaxThreads)
    residual_norm_kernel(const ResidualNormArgs a) {
  __shared__ float buf[2][1][16];
  int turn = 0;
  const int tpr = TPR ? TPR : blockDim.x, t = threadIdx.x % tpr;
  const int per = TPR ? kNormThreads / TPR : 1;
  float w[NV][V], wp[NV][V], sc[NV][V];
  load_weight<V, NV>(w, a.w, a.offset, 1.f, t, tpr, a.D);
  load_weight<V, NV>(wp, a.w_post, a.offset, 1.f, t, tpr, a.D);
  load_weight<V, NV>(sc, a.scale, 0.f, 1.f, t, tpr, a.D);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) wp[j][e] *= sc[j][e];
  const float inv = 1.f / float(a.D);
  constexpr int kStages = stages(2 * sizeof(T) + sizeof(TR));
  extern __shared__ __align__(16) unsigned char smem[];
  [[maybe_unused]] unsigned char* top = smem;
  [[maybe_unused]] const Ring<TR, V, NV, kStages> rr(top);
  [[maybe_unused]] const Ring<T, V, NV, kStages> rx(top);
  [[maybe_unused]] const Ring<T, V, NV, kStages> rz(top);
  const long long stride = (long long)gridDim.x * per;
  const int sub = threadIdx.x / tpr;
  const auto fetch = [&](int stage, long long row) {
    if constexpr (kStaged<NV, V>) {
      if (row < a.rows + per) {  // (a whole CTA's rows past the end: nothing to copy)
        const int D = row < a.rows ? a.D : 0;
        const size_t at = size_t(row < a.rows ? row : 0) * a.D;
        rx.fetch(stage, static_cast<const T*>(a.x) + at, t, tpr, D);
        rr.fetch(stage, static_cast<const TR*>(a.r) + at, t, tpr, D);
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
    Vec<T, V> x[NV], z[NV];
    Vec<TR, V> r[NV];
    if constexpr (kStaged<NV, V>) {
      copies_wait<kStages>();
      rx.take(x, stage);
      rr.take(r, stage);
      if (a.z) rz.take(z, stage);
      fetch(stage == 0 ? kStages - 1 : stage - 1, row + (kStages - 1) * stride);
      stage = stage == kStages - 1 ? 0 : stage + 1;
    } else {
      load_row<T, V, NV>(x, static_cast<const T*>(a.x) + at, t, tpr, D);
      load_row<TR, V, NV>(r, static_cast<const TR*>(a.r) + at, t, tpr, D);
      if (a.z) load_row<T, V, NV>(z, static_cast<const T*>(a.z) + at, t, tpr, D);
    }
    float rstd = 1.f;
    if (a.w_post) {
      float s[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) s[0] = fmaf(to_f(x[j].v[e]), to_f(x[j].v[e]), s[0]);
      row_sum<TPR, 1>(s, buf, turn);
      rstd = rsqrtf(fmaf(s[0], inv, a.eps));
    }
    float q[NV][V], s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float u = to_f(x[j].v[e]) * rstd * wp[j][e];
        if (a.z) u *= gate(a.act, to_f(z[j].v[e]));
        q[j][e] = to_f(r[j].v[e]) + u;
        s[0] = fmaf(q[j][e], q[j][e], s[0]);
      }
    store_row<TR, V, NV>(static_cast<TR*>(a.r_out) + at, q, t, tpr, D);
    row_sum<TPR, 1>(s, buf, turn);
    const float rs = rsqrtf(fmaf(s[0], inv, a.eps));
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) q[j][e] *= rs * w[j][e];
    store_row<T, V, NV>(static_cast<T*>(a.y) + at, q, t, tpr, D);
  }
}

template <int TPR, int NV, int V, typename T, typename TR>
__global__ void __launch_bounds__(TPR ? kNormThreads : kNormMaxThreads)
    residual_norm_backward_kernel(const ResidualNormArgs a) {
  __shared__ float buf3[2][3][16], buf1[2][1][16];
  __shared__ float groups[TPR ? kNormThreads * NV * V : 1];
  int turn3 = 0, turn1 = 0;
  const int tpr = TPR ? TPR : blockDim.x, t = threadIdx.x % tpr;
  const int per = TPR ? kNormThreads / TPR : 1;
  float w[NV][V], wp[NV][V], sc[NV][V], dw[NV][V], dwp[NV][V], dsc[NV][V];
  load_weight<V, NV>(w, a.w, a.offset, 1.f, t, tpr, a.D);
  load_weight<V, NV>(wp, a.w_post, a.offset, 1.f, t, tpr, a.D);
  load_weight<V, NV>(sc, a.scale, 0.f, 1.f, t, tpr, a.D);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[j][e] = dwp[j][e] = dsc[j][e] = 0.f;
  const float inv = 1.f / float(a.D);
  constexpr int kStages = stages(3 * sizeof(T) + 2 * sizeof(TR));
  extern __shared__ __align__(16) unsigned char smem[];
  [[maybe_unused]] unsigned char* top = smem;
  [[maybe_unused]] const Ring<TR, V, NV, kStages> rr(top);
  [[maybe_unused]] const Ring<TR, V, NV, kStages> rg(top);
  [[maybe_unused]] const Ring<T, V, NV, kStages> rd(top);
  [[maybe_unused]] const Ring<T, V, NV, kStages> rx(top);
  [[maybe_unused]] const Ring<T, V, NV, kStages> rz(top);
  const long long stride = (long long)gridDim.x * per;
  const int sub = threadIdx.x / tpr;
  const auto fetch = [&](int stage, long long row) {
    if constexpr (kStaged<NV, V>) {
      if (row < a.rows + per) {  // (a whole CTA's rows past the end: nothing to copy)
        const int D = row < a.rows ? a.D : 0;
        const size_t at = size_t(row < a.rows ? row : 0) * a.D;
        rr.fetch(stage, static_cast<const TR*>(a.r) + at, t, tpr, D);
        rd.fetch(stage, static_cast<const T*>(a.dy) + at, t, tpr, D);
        rx.fetch(stage, static_cast<const T*>(a.x) + at, t, tpr, D);
        if (a.dr_out) rg.fetch(stage, static_cast<const TR*>(a.dr_out) + at, t, tpr, D);
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
    Vec<T, V> x[NV], z[NV], dy[NV];
    Vec<TR, V> r[NV], dr[NV];
    if constexpr (kStaged<NV, V>) {
      copies_wait<kStages>();
      rr.take(r, stage);
      rd.take(dy, stage);
      rx.take(x, stage);
      if (a.dr_out) {
        rg.take(dr, stage);
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) dr[j] = Vec<TR, V>{};
      }
      if (a.z) rz.take(z, stage);
      fetch(stage == 0 ? kStages - 1 : stage - 1, row + (kStages - 1) * stride);
      stage = stage == kStages - 1 ? 0 : stage + 1;
    } else {
      load_row<TR, V, NV>(r, static_cast<const TR*>(a.r) + at, t, tpr, D);
      load_row<T, V, NV>(dy, static_cast<const T*>(a.dy) + at, t, tpr, D);
      load_row<T, V, NV>(x, static_cast<const T*>(a.x) + at, t, tpr, D);
      load_row<TR, V, NV>(dr, static_cast<const TR*>(a.dr_out) + at, t, tpr, a.dr_out ? D : 0);
      if (a.z) load_row<T, V, NV>(z, static_cast<const T*>(a.z) + at, t, tpr, D);
    }
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float re = to_f(r[j].v[e]), xe = to_f(x[j].v[e]);
        s[0] = fmaf(re, re, s[0]);
        s[1] = fmaf(to_f(dy[j].v[e]) * w[j][e], re, s[1]);
        s[2] = fmaf(xe, xe, s[2]);
      }
    row_sum<TPR, 3>(s, buf3, turn3);
    const float rs = rsqrtf(fmaf(s[0], inv, a.eps));
    const float c = s[1] * inv * rs * rs;
    const float rx = a.w_post ? rsqrtf(fmaf(s[2], inv, a.eps)) : 1.f;
    float q[NV][V], v[NV][V], dz[NV][V], m[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float re = to_f(r[j].v[e]), d = to_f(dy[j].v[e]);
        q[j][e] = fmaf(rs, fmaf(-c, re, d * w[j][e]), to_f(dr[j].v[e]));
        dw[j][e] = fmaf(d, re * rs, dw[j][e]);
        const float xh = to_f(x[j].v[e]) * rx, u = xh * wp[j][e];
        float av = 1.f, da = 0.f;
        if (a.z) gate_slope(a.act, to_f(z[j].v[e]), &av, &da);
        const float qa = q[j][e] * av;
        dsc[j][e] = fmaf(qa, u, dsc[j][e]);
        dz[j][e] = q[j][e] * sc[j][e] * u * da;
        v[j][e] = qa * sc[j][e];
        dwp[j][e] = fmaf(v[j][e], xh, dwp[j][e]);
        m[0] = fmaf(v[j][e], u, m[0]);
      }
    store_row<TR, V, NV>(static_cast<TR*>(a.dr) + at, q, t, tpr, D);
    if (a.z) store_row<T, V, NV>(static_cast<T*>(a.dz) + at, dz, t, tpr, D);
    if (a.w_post) {
      row_sum<TPR, 1>(m, buf1, turn1);
      const float k = m[0] * inv * rx;  // times x: xh mean(v w_post xh)
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e)
          v[j][e] = rx * fmaf(-k, to_f(x[j].v[e]), v[j][e] * wp[j][e]);
    }
    store_row<T, V, NV>(static_cast<T*>(a.dx) + at, v, t, tpr, D);
  }
  // partial gradients of the weights that there are: w, then w_post, then scale
  float* part = a.part + size_t(blockIdx.x) * a.D * a.weights;
  store_partial<TPR, V, NV>(part, dw, groups, t, tpr, a.D);
  if (a.w_post) store_partial<TPR, V, NV>(part += a.D, dwp, groups, t, tpr, a.D);
  if (a.scale) store_partial<TPR, V, NV>(part += a.D, dsc, groups, t, tpr, a.D);
}

// 32 columns a CTA; warp i adds the parts i, i + 8, ..., then the warps are added.
__global__ void __launch_bounds__(256)
    reduce_parts_kernel(const float* part, int n, int cols, float* d0, float* d1, float* d2, int D) {
  __shared__ float sum[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < cols)
    for (int p = w; p < n; p += 8) s += part[size_t(p) * cols + c];
  sum[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < cols) {
    for (int i = 1; i < 8; ++i) s += sum[i][lane];
    (c < D ? d0 : c < 2 * D ? d1 : d2)[c % D] = s;
  }
}

constexpr long long kForwardCtas = 2;  // per SM

template <typename T, typename TR>
struct Forward {
  const ResidualNormArgs& a;
  int sms;
  cudaStream_t stream;
  template <int TPR, int NV, int V>
  int run() {
    const int threads = norm_threads<TPR, NV, V>(a.D), per = TPR ? kNormThreads / TPR : 1;
    const long long groups = (a.rows + per - 1) / per;
    const int grid = int(groups < kForwardCtas * sms ? groups : kForwardCtas * sms);
    constexpr size_t kBytes = 2 * sizeof(T) + sizeof(TR);  // staged of a channel
    constexpr size_t kThread = kStaged<NV, V> ? stages(kBytes) * NV * V * kBytes : 0;
    constexpr int kMost = TPR ? kNormThreads : kNormMaxThreads;
    if (!raise_smem<&residual_norm_kernel<TPR, NV, V, T, TR>>(kThread * kMost)) return GDN_ERR_LAUNCH;
    residual_norm_kernel<TPR, NV, V, T, TR><<<grid, threads, kThread * threads, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
  }
};

template <typename T, typename TR>
struct Backward {
  const ResidualNormArgs& a;
  int sms;
  cudaStream_t stream;
  template <int TPR, int NV, int V>
  int run() {
    const int threads = norm_threads<TPR, NV, V>(a.D), per = TPR ? kNormThreads / TPR : 1;
    const long long groups = (a.rows + per - 1) / per;
    const int most = norm_max_parts(a.rows, a.D);
    const int grid = int(groups < most ? groups : most);
    constexpr size_t kBytes = 3 * sizeof(T) + 2 * sizeof(TR);  // staged of a channel
    constexpr size_t kThread = kStaged<NV, V> ? stages(kBytes) * NV * V * kBytes : 0;
    constexpr int kMost = TPR ? kNormThreads : kNormMaxThreads;
    if (!raise_smem<&residual_norm_backward_kernel<TPR, NV, V, T, TR>>(kThread * kMost)) return GDN_ERR_LAUNCH;
    residual_norm_backward_kernel<TPR, NV, V, T, TR><<<grid, threads, kThread * threads, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_LAUNCH;
    float* dst[3] = {a.dw, a.w_post ? a.dw_post : a.dscale, a.dscale};
    return launch_reduce_parts(a.part, grid, a.D * a.weights, dst, a.D, stream);
  }
};

bool wide_ok(const ResidualNormArgs& a) {
  const void* p[] = {a.x, a.r, a.z, a.w, a.w_post, a.scale, a.y, a.r_out, a.dy, a.dr_out,
                     a.dx, a.dr, a.dz, a.part};
  uintptr_t all = 0;
  for (const void* q : p) all |= reinterpret_cast<uintptr_t>(q);
  return (all & 15) == 0;
}

template <template <typename, typename> class Run>
int dispatch(const ResidualNormArgs& a, int dtype, int r_dtype, int sms, cudaStream_t stream) {
  using B = __nv_bfloat16;
  const bool wide = wide_ok(a);
  if (dtype == GDN_F32) return with_layout(a.D, wide, Run<float, float>{a, sms, stream});
  return r_dtype == GDN_BF16 ? with_layout(a.D, wide, Run<B, B>{a, sms, stream})
                             : with_layout(a.D, wide, Run<B, float>{a, sms, stream});
}

}  // namespace

int launch_reduce_parts(const float* part, int n, int cols, float* const* dst, int D,
                        cudaStream_t stream) {
  const int weights = cols / D;
  reduce_parts_kernel<<<(cols + 31) / 32, 256, 0, stream>>>(
      part, n, cols, dst[0], weights > 1 ? dst[1] : nullptr, weights > 2 ? dst[2] : nullptr, D);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

int launch_residual_norm(const ResidualNormArgs& a, int dtype, int r_dtype, int sms,
                         cudaStream_t stream) {
  return dispatch<Forward>(a, dtype, r_dtype, sms, stream);
}

int launch_residual_norm_backward(const ResidualNormArgs& a, int dtype, int r_dtype, int sms,
                                  cudaStream_t stream) {
  return dispatch<Backward>(a, dtype, r_dtype, sms, stream);
}

}  // namespace gdn
