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
#include "gdn_norm.cuh"

namespace gdn {
namespace {

template <typename L, typename T, typename TR>
__global__ void __launch_bounds__(L::TH) residual_norm_kernel(const ResidualNormArgs a) {
  constexpr int kAll = 2 * sizeof(T) + sizeof(TR), kStages = stages(kAll), P = L::P, N = L::N;
  using RR = Ring<L, TR, 0, kAll>;
  using RX = Ring<L, T, sizeof(TR), kAll>;
  using RZ = Ring<L, T, sizeof(TR) + sizeof(T), kAll>;
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
      RX::fetch(smem, to, static_cast<const T*>(a.x) + o, at, on);
      RR::fetch(smem, to, static_cast<const TR*>(a.r) + o, at, on);
      if (a.z) RZ::fetch(smem, to, static_cast<const T*>(a.z) + o, at, on);
    }
    copies_commit();
    next += stride;
    to = to == kStages - 1 ? 0 : to + 1;
  };
  if constexpr (L::kStaged) {
    RR::clear(smem, at);
    RX::clear(smem, at);
    RZ::clear(smem, at);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch();
  }
  F<P> w[N], wp[N];  // wp: the post norm's weight times the scale
  load_weight<L>(w, a.scale, 0.f, at);
  load_weight<L>(wp, a.w_post, a.offset, at);
#pragma unroll
  for (int i = 0; i < N; ++i) wp[i] = mul(wp[i], w[i]);
  load_weight<L>(w, a.w, a.offset, at);
  const float inv = 1.f / float(a.D);
  for (; row - at.sub < a.rows; row += stride) {
    const bool on = !L::kShort || row < a.rows;
    const size_t o = size_t(on ? row : 0) * a.D;
    F<P> x[N], r[N], z[N];
    if constexpr (L::kStaged) {
      copies_wait<kStages>();
      RX::take(x, smem, stage);
      RR::take(r, smem, stage);
      if (a.z) RZ::take(z, smem, stage);
      stage = stage == kStages - 1 ? 0 : stage + 1;
      fetch();
    } else {
      load_row<L, T>(x, static_cast<const T*>(a.x) + o, at, on);
      load_row<L, TR>(r, static_cast<const TR*>(a.r) + o, at, on);
      if (a.z) load_row<L, T>(z, static_cast<const T*>(a.z) + o, at, on);
    }
    float rstd = 1.f;
    if (a.w_post) {
      F<P> sq = all<P>(0.f);
#pragma unroll
      for (int i = 0; i < N; ++i) sq = fma(x[i], x[i], sq);
      float s[1] = {total(sq)};
      row_sum<L, 1>(s, buf, turn);
      rstd = rsqrtf(fmaf(s[0], inv, a.eps));
    }
    F<P> sq = all<P>(0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = mul(x[i], all<P>(rstd));
      if (a.z) x[i] = mul(x[i], gate(a.act, z[i]));
      r[i] = fma(x[i], wp[i], r[i]);
      sq = fma(r[i], r[i], sq);
    }
    store_row<L, TR>(static_cast<TR*>(a.r_out) + o, r, at, on);
    float s[1] = {total(sq)};
    row_sum<L, 1>(s, buf, turn);
    const F<P> rs = all<P>(rsqrtf(fmaf(s[0], inv, a.eps)));
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = mul(mul(r[i], rs), w[i]);
    store_row<L, T>(static_cast<T*>(a.y) + o, r, at, on);
  }
}

template <typename L, typename T, typename TR>
__global__ void __launch_bounds__(L::TH) residual_norm_backward_kernel(const ResidualNormArgs a) {
  constexpr int kT = sizeof(T), kR = sizeof(TR), kAll = 3 * kT + 2 * kR, kStages = stages(kAll);
  constexpr int P = L::P, N = L::N;
  using RR = Ring<L, TR, 0, kAll>;
  using RG = Ring<L, TR, kR, kAll>;
  using RD = Ring<L, T, 2 * kR, kAll>;
  using RX = Ring<L, T, 2 * kR + kT, kAll>;
  using RZ = Ring<L, T, 2 * kR + 2 * kT, kAll>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ SumBuffer<L, 3> buf3;
  __shared__ SumBuffer<L, 1> buf1;
  __shared__ float groups[L::kShort ? L::TH * L::NV * L::V : 1];
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
  if constexpr (L::kStaged) {
    RR::clear(smem, at);
    RG::clear(smem, at);
    RD::clear(smem, at);
    RX::clear(smem, at);
    RZ::clear(smem, at);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch();
  }
  F<P> w[N], wp[N], sc[N], dw[N], dwp[N], dsc[N];
  load_weight<L>(w, a.w, a.offset, at);
  load_weight<L>(wp, a.w_post, a.offset, at);
  load_weight<L>(sc, a.scale, 0.f, at);
#pragma unroll
  for (int i = 0; i < N; ++i) dw[i] = dwp[i] = dsc[i] = all<P>(0.f);
  const float inv = 1.f / float(a.D);
  for (; row - at.sub < a.rows; row += stride) {
    const bool on = !L::kShort || row < a.rows;
    const size_t o = size_t(on ? row : 0) * a.D;
    F<P> x[N], z[N], dy[N], r[N], q[N];
    if constexpr (L::kStaged) {
      copies_wait<kStages>();
      RR::take(r, smem, stage);
      RD::take(dy, smem, stage);
      RX::take(x, smem, stage);
      if (a.dr_out) RG::take(q, smem, stage);
      if (a.z) RZ::take(z, smem, stage);
      stage = stage == kStages - 1 ? 0 : stage + 1;
      fetch();
    } else {
      load_row<L, TR>(r, static_cast<const TR*>(a.r) + o, at, on);
      load_row<L, T>(dy, static_cast<const T*>(a.dy) + o, at, on);
      load_row<L, T>(x, static_cast<const T*>(a.x) + o, at, on);
      if (a.dr_out) load_row<L, TR>(q, static_cast<const TR*>(a.dr_out) + o, at, on);
      if (a.z) load_row<L, T>(z, static_cast<const T*>(a.z) + o, at, on);
    }
    if (!a.dr_out) {
#pragma unroll
      for (int i = 0; i < N; ++i) q[i] = all<P>(0.f);
    }
    F<P> s0 = all<P>(0.f), s1 = s0, s2 = s0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s0 = fma(r[i], r[i], s0);
      s1 = fma(mul(dy[i], w[i]), r[i], s1);
      s2 = fma(x[i], x[i], s2);
    }
    float s[3] = {total(s0), total(s1), total(s2)};
    row_sum<L, 3>(s, buf3, turn3);
    const float rs = rsqrtf(fmaf(s[0], inv, a.eps));
    const float rx = a.w_post ? rsqrtf(fmaf(s[2], inv, a.eps)) : 1.f;
    const F<P> rr = all<P>(rs), c = all<P>(-(s[1] * inv * rs * rs)), rp = all<P>(rx);
    F<P> sm = all<P>(0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      q[i] = fma(rr, fma(c, r[i], mul(dy[i], w[i])), q[i]);
      dw[i] = fma(dy[i], mul(r[i], rr), dw[i]);
      x[i] = mul(x[i], rp);  // xh
      const F<P> u = mul(x[i], wp[i]);
      F<P> qa = q[i];
      if (a.z) {
        F<P> av, da;
        gate_slope(a.act, z[i], &av, &da);
        qa = mul(qa, av);
        z[i] = mul(mul(mul(q[i], sc[i]), u), da);  // dz
      }
      dsc[i] = fma(qa, u, dsc[i]);
      r[i] = mul(qa, sc[i]);  // v
      dwp[i] = fma(r[i], x[i], dwp[i]);
      sm = fma(r[i], u, sm);
    }
    store_row<L, TR>(static_cast<TR*>(a.dr) + o, q, at, on);
    if (a.z) store_row<L, T>(static_cast<T*>(a.dz) + o, z, at, on);
    if (a.w_post) {
      float m[1] = {total(sm)};
      row_sum<L, 1>(m, buf1, turn1);
      const F<P> k = all<P>(-(m[0] * inv));  // -mean(v w_post xh)
#pragma unroll
      for (int i = 0; i < N; ++i) r[i] = mul(rp, fma(k, x[i], mul(r[i], wp[i])));
    }
    store_row<L, T>(static_cast<T*>(a.dx) + o, r, at, on);
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // partial gradients of the weights that there are: w, then w_post, then scale
  float* part = a.part + size_t(blockIdx.x) * a.D * a.weights;
  store_partial<L>(part, dw, groups, at);
  if (a.w_post) store_partial<L>(part += a.D, dwp, groups, at);
  if (a.scale) store_partial<L>(part += a.D, dsc, groups, at);
}

// 32 columns a CTA; warp i adds the parts i, i + 32, ..., then the warps are added.
// The launch may start before the parts are complete: it waits for the launch
// before it first.
constexpr int kReduceWarps = 32;
__global__ void __launch_bounds__(32 * kReduceWarps)
    reduce_parts_kernel(const float* part, int n, int cols, float* d0, float* d1, float* d2, int D) {
  __shared__ float sum[kReduceWarps][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 10
    for (int p = w; p < n; p += kReduceWarps) s += part[size_t(p) * cols + c];
  }
  sum[w][lane] = s;
  __syncthreads();
  // warp w adds column w: lane i has the sum of warp i
  s = sum[lane][w];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int col = blockIdx.x * 32 + w;
  if (lane == 0 && col < cols) (col < D ? d0 : col < 2 * D ? d1 : d2)[col % D] = s;
}

constexpr long long kForwardCtas = 4;  // per SM

template <typename T, typename TR>
struct Forward {
  const ResidualNormArgs& a;
  int sms;
  cudaStream_t stream;
  template <typename L>
  int run() {
    const long long groups = (a.rows + L::kRows - 1) / L::kRows;
    const int grid = int(std::min(groups, kForwardCtas * sms));
    constexpr size_t smem = ring_bytes<L>(2 * sizeof(T) + sizeof(TR));
    if (!raise_smem<&residual_norm_kernel<L, T, TR>>(smem)) return GDN_ERR_LAUNCH;
    residual_norm_kernel<L, T, TR><<<grid, L::TH, smem, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
  }
  int run4096() { return run<Layout<256, 256, 4, 4>>(); }
};

template <typename T, typename TR>
struct Backward {
  const ResidualNormArgs& a;
  int sms;
  cudaStream_t stream;
  template <typename L>
  int run() {
    const long long groups = (a.rows + L::kRows - 1) / L::kRows;
    const int grid = int(std::min<long long>(groups, norm_max_parts(a.rows, a.D)));
    constexpr size_t smem = ring_bytes<L>(3 * sizeof(T) + 2 * sizeof(TR));
    if (!raise_smem<&residual_norm_backward_kernel<L, T, TR>>(smem)) return GDN_ERR_LAUNCH;
    residual_norm_backward_kernel<L, T, TR><<<grid, L::TH, smem, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_LAUNCH;
    float* dst[3] = {a.dw, a.w_post ? a.dw_post : a.dscale, a.dscale};
    return launch_reduce_parts(a.part, grid, a.D * a.weights, dst, a.D, stream);
  }
  int run4096() { return run<Layout<512, 512, 2, 4>>(); }
};

// Whether every array starts on four elements.
bool wide_ok(const ResidualNormArgs& a, int dtype, int r_dtype) {
  const uintptr_t e = dtype == GDN_BF16 ? 8 : 16, er = r_dtype == GDN_BF16 ? 8 : 16;
  return aligned(a.x, e) && aligned(a.z, e) && aligned(a.y, e) && aligned(a.dy, e) &&
         aligned(a.dx, e) && aligned(a.dz, e) && aligned(a.r, er) && aligned(a.r_out, er) &&
         aligned(a.dr_out, er) && aligned(a.dr, er) && aligned(a.w, 16) && aligned(a.w_post, 16) &&
         aligned(a.scale, 16);
}

template <template <typename, typename> class Run>
int dispatch(const ResidualNormArgs& a, int dtype, int r_dtype, int sms, cudaStream_t stream) {
  using B = __nv_bfloat16;
  const bool wide = wide_ok(a, dtype, r_dtype);
  if (dtype == GDN_F32) return with_layout(a.D, wide, Run<float, float>{a, sms, stream});
  return r_dtype == GDN_BF16 ? with_layout(a.D, wide, Run<B, B>{a, sms, stream})
                             : with_layout(a.D, wide, Run<B, float>{a, sms, stream});
}

}  // namespace

int launch_reduce_parts(const float* part, int n, int cols, float* const* dst, int D,
                        cudaStream_t stream) {
  const int weights = cols / D;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((cols + 31) / 32);
  cfg.blockDim = dim3(32 * kReduceWarps);
  cfg.stream = stream;
  cudaLaunchAttribute at{};  // its start overlaps the end of the launch before it
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, &reduce_parts_kernel, part, n, cols, dst[0],
                            weights > 1 ? dst[1] : static_cast<float*>(nullptr),
                            weights > 2 ? dst[2] : static_cast<float*>(nullptr), D) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_LAUNCH;
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
