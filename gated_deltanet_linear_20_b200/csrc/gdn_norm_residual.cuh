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
//
// The two directions are files of their own, which compile side by side.
#pragma once

#include "gdn_norm.cuh"

namespace gdn {

// How many elements every array starts on a multiple of: 4, 2 or 1.
inline int width(const ResidualNormArgs& a, int dtype, int r_dtype) {
  const uintptr_t e = dtype == GDN_BF16 ? 2 : 4, er = r_dtype == GDN_BF16 ? 2 : 4;
  const auto ok = [&](uintptr_t n) {
    return aligned(a.x, n * e) && aligned(a.z, n * e) && aligned(a.y, n * e) &&
           aligned(a.dy, n * e) && aligned(a.dx, n * e) && aligned(a.dz, n * e) &&
           aligned(a.r, n * er) && aligned(a.r_out, n * er) && aligned(a.dr_out, n * er) &&
           aligned(a.dr, n * er) && aligned(a.w, n * 4) && aligned(a.w_post, n * 4) &&
           aligned(a.scale, n * 4);
  };
  return ok(4) ? 4 : ok(2) ? 2 : 1;
}

template <template <typename, typename> class Run, int LONG, bool TRIM>
int dispatch(const ResidualNormArgs& a, int dtype, int r_dtype, int sms, cudaStream_t stream) {
  using B = __nv_bfloat16;
  const int n = width(a, dtype, r_dtype);
  if (dtype == GDN_F32) return with_layout<LONG, TRIM>(a.D, n, Run<float, float>{a, sms, stream});
  return r_dtype == GDN_BF16 ? with_layout<LONG, TRIM>(a.D, n, Run<B, B>{a, sms, stream})
                             : with_layout<LONG, TRIM>(a.D, n, Run<B, float>{a, sms, stream});
}

}  // namespace gdn
