// C-ABI entry points of the channel recurrence and of the norms: argument
// checks, then the launches on the caller's stream.
#include <cmath>

#include "gdn_host.h"
#include "gdn_internal.h"

namespace {

using gdn::aligned;
using gdn::Span;

constexpr long long kMaxTokens = 1LL << 30;
constexpr long long kMaxElements = 1LL << 38;  // more than the device holds

int elem_size(int dtype) { return dtype == GDN_BF16 ? 2 : dtype == GDN_F32 ? 4 : 0; }

long long carry_rows(long long N, long long tokens, bool packed) {
  if (packed) return tokens / GDN_SCAN_CARRY_TOKENS + N;
  const long long T = N > 0 ? tokens / N : 0;
  return N * ((T + GDN_SCAN_CARRY_TOKENS - 1) / GDN_SCAN_CARRY_TOKENS);
}

// Sizes shared by the scan calls.  *done: nothing to do (GDN_OK is returned).
int scan_sizes(long long N, long long tokens, int C, int dtype, bool* done) {
  *done = false;
  if (N < 0 || tokens < 0 || C < 0) return GDN_ERR_SHAPE;
  if (!elem_size(dtype)) return GDN_ERR_UNSUPPORTED;
  if (tokens > kMaxTokens || N > kMaxTokens || (tokens + N) * C > kMaxElements) return GDN_ERR_SHAPE;
  *done = N == 0 || C == 0;
  return GDN_OK;
}

int scan_impl(gdn::ScanArgs a, long long tokens, int dtype, void* stream) {
  bool done;
  int rc = scan_sizes(a.N, tokens, a.C, dtype, &done);
  if (rc != GDN_OK || done) return rc;
  const size_t e = elem_size(dtype), act = size_t(tokens) * a.C, st = size_t(a.N) * a.C * 4;
  if (!a.h_T || (tokens > 0 && (!a.x || !a.g || !a.h))) return GDN_ERR_NULL;
  if (!aligned(a.x, e) || !aligned(a.beta, e) || !aligned(a.h, e) || !aligned(a.g, 4) ||
      !aligned(a.h0, 4) || !aligned(a.h_T, 4) || !aligned(a.carries, 4) ||
      !aligned(a.cu_seqlens, 4) || !aligned(a.status, 4))
    return GDN_ERR_ALIGN;
  const size_t cb = size_t(carry_rows(a.N, tokens, a.cu_seqlens != nullptr)) * a.C * 4;
  const Span ins[] = {{a.h0, st}, {a.x, act * e}, {a.g, act * 4}, {a.beta, act * e},
                      {a.cu_seqlens, (size_t(a.N) + 1) * 4}};
  const Span outs[] = {{a.h_T, st}, {a.h, act * e}, {a.carries, cb}, {a.status, 4}};
  const int same[] = {0, -1, -1, -1};  // h_T may be h0
  if (gdn::any_alias(outs, 4, ins, 5, same)) return GDN_ERR_ALIAS;
  int sms = 0;
  rc = gdn::require_device(&sms);
  if (rc != GDN_OK) return rc;
  return gdn::launch_scan(a, dtype, sms, static_cast<cudaStream_t>(stream));
}

int scan_backward_impl(gdn::ScanBackwardArgs b, int carries_valid, long long tokens, int dtype,
                       void* stream) {
  gdn::ScanArgs& a = b.f;
  bool done;
  int rc = scan_sizes(a.N, tokens, a.C, dtype, &done);
  if (rc != GDN_OK || done) return rc;
  const size_t e = elem_size(dtype), act = size_t(tokens) * a.C, st = size_t(a.N) * a.C * 4;
  if (tokens > 0 && (!a.x || !a.g || !b.dh || !b.dx || !b.dg || !a.carries ||
                     (a.beta != nullptr) != (b.dbeta != nullptr)))
    return GDN_ERR_NULL;
  if (!aligned(a.x, e) || !aligned(a.beta, e) || !aligned(b.dh, e) || !aligned(b.dx, e) ||
      !aligned(b.dbeta, e) || !aligned(a.g, 4) || !aligned(b.dg, 4) || !aligned(a.h0, 4) ||
      !aligned(b.dh_T, 4) || !aligned(b.dh0, 4) || !aligned(a.carries, 4) ||
      !aligned(a.cu_seqlens, 4) || !aligned(a.status, 4))
    return GDN_ERR_ALIGN;
  const size_t cb = size_t(carry_rows(a.N, tokens, a.cu_seqlens != nullptr)) * a.C * 4;
  const Span ins[] = {{b.dh_T, st}, {a.x, act * e}, {a.g, act * 4}, {a.beta, act * e},
                      {a.h0, st}, {b.dh, act * e}, {a.cu_seqlens, (size_t(a.N) + 1) * 4}};
  const Span outs[] = {{b.dh0, st}, {b.dx, act * e}, {b.dg, act * 4}, {b.dbeta, act * e},
                       {a.carries, cb}, {a.status, 4}};
  const int same[] = {0, -1, -1, -1, -1, -1};  // dh0 may be dh_T
  if (gdn::any_alias(outs, 6, ins, 7, same)) return GDN_ERR_ALIAS;
  int sms = 0;
  rc = gdn::require_device(&sms);
  if (rc != GDN_OK) return rc;
  const cudaStream_t st_ = static_cast<cudaStream_t>(stream);
  if (!carries_valid && tokens > 0) {  // the states alone: no h, no h_T
    gdn::ScanArgs f = a;
    f.h = nullptr;
    f.h_T = nullptr;
    rc = gdn::launch_scan(f, dtype, sms, st_);
    if (rc != GDN_OK) return rc;
  }
  return gdn::launch_scan_backward(b, dtype, sms, st_);
}

// Reads the norm options (NULL: defaults); false if they are invalid.
bool read_norm_options(const gdn_norm_options* o, float* eps, float* offset, int* gate) {
  *eps = 1e-6f;
  *offset = 0.f;
  *gate = GDN_GATE_SILU;
  if (!o) return true;
  if (o->size < int(sizeof(gdn_norm_options))) return false;
  *eps = o->eps;
  *offset = o->weight_offset;
  *gate = o->gate;
  return std::isfinite(*eps) && *eps >= 0.f && std::isfinite(*offset) &&
         (*gate == GDN_GATE_SILU || *gate == GDN_GATE_SIGMOID);
}

int norm_sizes(long long rows, int D) {
  if (rows < 0 || D < 0 || D > gdn::kNormMaxD || rows * D > kMaxElements) return GDN_ERR_SHAPE;
  return GDN_OK;
}

size_t norm_workspace(int rows, int D, int weights) {
  if (rows <= 0 || D <= 0 || D > gdn::kNormMaxD || weights < 1 || weights > 3) return 0;
  return size_t(gdn::norm_max_parts(rows, D)) * D * weights * 4;
}

int check_workspace(const void* ws, size_t have, size_t need) {
  return !ws || !aligned(ws, 256) || have < need ? GDN_ERR_WORKSPACE : GDN_OK;
}

}  // namespace

extern "C" {

size_t gdn_scan_carry_bytes(int N, int tokens, int C, int packed) {
  if (N < 0 || tokens < 0 || C < 0) return 0;
  return size_t(carry_rows(N, tokens, packed != 0)) * size_t(C) * 4;
}

int gdn_scan(const void* x, const float* g, const void* beta, const float* h0, void* h, float* h_T,
             float* carries, int B, int T, int C, int dtype, int* status, void* stream) {
  if (B < 0 || T < 0) return GDN_ERR_SHAPE;
  return scan_impl({x, g, beta, h0, h, h_T, carries, nullptr, B, T, C, 0, status},
                   (long long)B * T, dtype, stream);
}

int gdn_scan_varlen(const void* x, const float* g, const void* beta, const float* h0, void* h,
                    float* h_T, float* carries, const int* cu_seqlens, int N, int total_T, int C,
                    int dtype, int* status, void* stream) {
  if (N > 0 && C > 0 && total_T >= 0 && !cu_seqlens) return GDN_ERR_NULL;
  return scan_impl({x, g, beta, h0, h, h_T, carries, cu_seqlens, N, total_T, C, 0, status},
                   total_T, dtype, stream);
}

int gdn_scan_step(const void* x, const float* g, const void* beta, float* state, void* h, int B,
                  int C, int dtype, void* stream) {
  bool done;
  int rc = scan_sizes(B, B, C, dtype, &done);
  if (rc != GDN_OK || done) return rc;
  const size_t e = elem_size(dtype), n = size_t(B) * C;
  if (!x || !g || !state || !h) return GDN_ERR_NULL;
  if (!aligned(x, e) || !aligned(beta, e) || !aligned(h, e) || !aligned(g, 4) || !aligned(state, 4))
    return GDN_ERR_ALIGN;
  const Span ins[] = {{x, n * e}, {g, n * 4}, {beta, n * e}};
  const Span outs[] = {{state, n * 4}, {h, n * e}};
  const int same[] = {-1, -1};
  if (gdn::any_alias(outs, 2, ins, 3, same)) return GDN_ERR_ALIAS;
  int sms = 0;
  rc = gdn::require_device(&sms);
  if (rc != GDN_OK) return rc;
  return gdn::launch_scan_step({x, g, beta, nullptr, h, state, nullptr, nullptr, B, 1, C, 0, nullptr},
                               dtype, static_cast<cudaStream_t>(stream));
}

int gdn_scan_backward(const void* x, const float* g, const void* beta, const float* h0,
                      const void* dh, const float* dh_T, void* dx, float* dg, void* dbeta,
                      float* dh0, float* carries, int carries_valid, int B, int T, int C,
                      int dtype, int* status, void* stream) {
  if (B < 0 || T < 0) return GDN_ERR_SHAPE;
  return scan_backward_impl(
      {{x, g, beta, h0, nullptr, nullptr, carries, nullptr, B, T, C, 0, status}, dh, dh_T, dx, dg,
       dbeta, dh0},
      carries_valid, (long long)B * T, dtype, stream);
}

int gdn_scan_varlen_backward(const void* x, const float* g, const void* beta, const float* h0,
                             const void* dh, const float* dh_T, void* dx, float* dg, void* dbeta,
                             float* dh0, float* carries, int carries_valid, const int* cu_seqlens,
                             int N, int total_T, int C, int dtype, int* status, void* stream) {
  if (N > 0 && C > 0 && total_T >= 0 && !cu_seqlens) return GDN_ERR_NULL;
  bool none;
  const int rc = scan_sizes(N, total_T, C, dtype, &none);
  if (rc == GDN_OK && N == 0) {  // tokens of no sequence: gradients of zero
    const size_t act = size_t(total_T) * C, e = elem_size(dtype);
    const Span grads[] = {{dx, act * e}, {dg, act * 4}, {dbeta, act * e}};
    for (const Span& d : grads)
      if (d.p && d.bytes && cudaMemsetAsync(const_cast<void*>(d.p), 0, d.bytes,
                                            static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    return GDN_OK;
  }
  return scan_backward_impl(
      {{x, g, beta, h0, nullptr, nullptr, carries, cu_seqlens, N, total_T, C, 0, status}, dh, dh_T,
       dx, dg, dbeta, dh0},
      carries_valid, total_T, dtype, stream);
}

size_t gdn_norm_workspace_bytes(int rows, int D, int weights) {
  return norm_workspace(rows, D, weights);
}

int gdn_gated_norm(const void* x, int x_dtype, const float* w, const void* z, void* y, int rows,
                   int D, int dtype, const gdn_norm_options* opts, void* stream) {
  gdn::GatedNormArgs a{};
  int rc = norm_sizes(rows, D);
  if (rc != GDN_OK) return rc;
  const size_t ex = elem_size(x_dtype), e = elem_size(dtype), n = size_t(rows) * D;
  if (!ex || !e || !read_norm_options(opts, &a.eps, &a.offset, &a.act)) return GDN_ERR_UNSUPPORTED;
  if (n == 0) return GDN_OK;
  if (!x || !w || !y) return GDN_ERR_NULL;
  if (!aligned(x, ex) || !aligned(z, e) || !aligned(y, e) || !aligned(w, 4)) return GDN_ERR_ALIGN;
  const Span ins[] = {{x, n * ex}, {z, n * e}, {w, size_t(D) * 4}};
  const Span outs[] = {{y, n * e}};
  const int same[] = {-1};
  if (gdn::any_alias(outs, 1, ins, 3, same)) return GDN_ERR_ALIAS;
  int sms = 0;
  rc = gdn::require_device(&sms);
  if (rc != GDN_OK) return rc;
  a.x = x;
  a.z = z;
  a.w = w;
  a.y = y;
  a.rows = rows;
  a.D = D;
  return gdn::launch_gated_norm(a, x_dtype, dtype, sms, static_cast<cudaStream_t>(stream));
}

int gdn_gated_norm_backward(const void* dy, const void* x, int x_dtype, const float* w,
                            const void* z, void* dx, void* dz, float* dw, int rows, int D,
                            int dtype, void* workspace, size_t workspace_bytes,
                            const gdn_norm_options* opts, void* stream) {
  gdn::GatedNormArgs a{};
  int rc = norm_sizes(rows, D);
  if (rc != GDN_OK) return rc;
  const size_t ex = elem_size(x_dtype), e = elem_size(dtype), n = size_t(rows) * D;
  if (!ex || !e || !read_norm_options(opts, &a.eps, &a.offset, &a.act)) return GDN_ERR_UNSUPPORTED;
  if (D == 0) return GDN_OK;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t wb = size_t(D) * 4, need = norm_workspace(rows, D, 1);
  if (!dw || (rows > 0 && (!dy || !x || !w || !dx || (z != nullptr) != (dz != nullptr))))
    return GDN_ERR_NULL;
  if (!aligned(x, ex) || !aligned(dx, ex) || !aligned(z, e) || !aligned(dy, e) || !aligned(dz, e) ||
      !aligned(w, 4) || !aligned(dw, 4))
    return GDN_ERR_ALIGN;
  if (rows > 0 && (rc = check_workspace(workspace, workspace_bytes, need)) != GDN_OK) return rc;
  const Span ins[] = {{dy, n * e}, {x, n * ex}, {z, n * e}, {w, wb}};
  const Span outs[] = {{dx, n * ex}, {dz, n * e}, {dw, wb}, {workspace, need}};
  const int same[] = {-1, -1, -1, -1};
  if (gdn::any_alias(outs, 4, ins, 4, same)) return GDN_ERR_ALIAS;
  int sms = 0;
  rc = gdn::require_device(&sms);
  if (rc != GDN_OK) return rc;
  if (rows == 0)
    return cudaMemsetAsync(dw, 0, wb, st) == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
  a.x = x;
  a.z = z;
  a.w = w;
  a.rows = rows;
  a.D = D;
  a.dy = dy;
  a.dx = dx;
  a.dz = dz;
  a.dw = dw;
  a.part = static_cast<float*>(workspace);
  return gdn::launch_gated_norm_backward(a, x_dtype, dtype, sms, st);
}

int gdn_residual_norm(const void* x, const void* r, const float* w, const void* z,
                      const float* w_post, const float* scale, void* y, void* r_out, int rows,
                      int D, int dtype, int r_dtype, const gdn_norm_options* opts, void* stream) {
  gdn::ResidualNormArgs a{};
  int rc = norm_sizes(rows, D);
  if (rc != GDN_OK) return rc;
  const size_t er = elem_size(r_dtype), e = elem_size(dtype), n = size_t(rows) * D;
  if (!er || !e || er < e || !read_norm_options(opts, &a.eps, &a.offset, &a.act))
    return GDN_ERR_UNSUPPORTED;
  if (n == 0) return GDN_OK;
  if (!x || !r || !w || !y || !r_out) return GDN_ERR_NULL;
  if (!aligned(x, e) || !aligned(z, e) || !aligned(y, e) || !aligned(r, er) ||
      !aligned(r_out, er) || !aligned(w, 4) || !aligned(w_post, 4) || !aligned(scale, 4))
    return GDN_ERR_ALIGN;
  const size_t wb = size_t(D) * 4;
  const Span ins[] = {{r, n * er}, {x, n * e}, {z, n * e}, {w, wb}, {w_post, wb}, {scale, wb}};
  const Span outs[] = {{r_out, n * er}, {y, n * e}};
  const int same[] = {0, -1};  // r_out may be r
  if (gdn::any_alias(outs, 2, ins, 6, same)) return GDN_ERR_ALIAS;
  int sms = 0;
  rc = gdn::require_device(&sms);
  if (rc != GDN_OK) return rc;
  a.x = x;
  a.r = r;
  a.z = z;
  a.w = w;
  a.w_post = w_post;
  a.scale = scale;
  a.y = y;
  a.r_out = r_out;
  a.rows = rows;
  a.D = D;
  return gdn::launch_residual_norm(a, dtype, r_dtype, sms, static_cast<cudaStream_t>(stream));
}

int gdn_residual_norm_backward(const void* dy, const void* dr_out, const void* x,
                               const void* r_out, const float* w, const void* z,
                               const float* w_post, const float* scale, void* dx, void* dr,
                               void* dz, float* dw, float* dw_post, float* dscale, int rows, int D,
                               int dtype, int r_dtype, void* workspace, size_t workspace_bytes,
                               const gdn_norm_options* opts, void* stream) {
  gdn::ResidualNormArgs a{};
  int rc = norm_sizes(rows, D);
  if (rc != GDN_OK) return rc;
  const size_t er = elem_size(r_dtype), e = elem_size(dtype), n = size_t(rows) * D;
  if (!er || !e || er < e || !read_norm_options(opts, &a.eps, &a.offset, &a.act))
    return GDN_ERR_UNSUPPORTED;
  if (D == 0) return GDN_OK;
  if (!dw || (w_post != nullptr) != (dw_post != nullptr) || (scale != nullptr) != (dscale != nullptr) ||
      (rows > 0 && (!dy || !x || !r_out || !w || !dx || !dr || (z != nullptr) != (dz != nullptr))))
    return GDN_ERR_NULL;
  if (!aligned(x, e) || !aligned(z, e) || !aligned(dy, e) || !aligned(dx, e) || !aligned(dz, e) ||
      !aligned(r_out, er) || !aligned(dr_out, er) || !aligned(dr, er) || !aligned(w, 4) ||
      !aligned(w_post, 4) || !aligned(scale, 4) || !aligned(dw, 4) || !aligned(dw_post, 4) ||
      !aligned(dscale, 4))
    return GDN_ERR_ALIGN;
  a.weights = 1 + (w_post ? 1 : 0) + (scale ? 1 : 0);
  const size_t wb = size_t(D) * 4, need = norm_workspace(rows, D, a.weights);
  if (rows > 0 && (rc = check_workspace(workspace, workspace_bytes, need)) != GDN_OK) return rc;
  const Span ins[] = {{dr_out, n * er}, {dy, n * e}, {x, n * e}, {r_out, n * er}, {z, n * e},
                      {w, wb}, {w_post, wb}, {scale, wb}};
  const Span outs[] = {{dr, n * er}, {dx, n * e}, {dz, n * e}, {dw, wb}, {dw_post, wb},
                       {dscale, wb}, {workspace, need}};
  const int same[] = {0, -1, -1, -1, -1, -1, -1};  // dr may be dr_out
  if (gdn::any_alias(outs, 7, ins, 8, same)) return GDN_ERR_ALIAS;
  int sms = 0;
  rc = gdn::require_device(&sms);
  if (rc != GDN_OK) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {  // no rows: gradients of zero
    float* const grads[] = {dw, dw_post, dscale};
    for (float* d : grads)
      if (d && cudaMemsetAsync(d, 0, wb, st) != cudaSuccess) return GDN_ERR_LAUNCH;
    return GDN_OK;
  }
  a.x = x;
  a.r = r_out;
  a.z = z;
  a.w = w;
  a.w_post = w_post;
  a.scale = scale;
  a.rows = rows;
  a.D = D;
  a.dy = dy;
  a.dr_out = dr_out;
  a.dx = dx;
  a.dr = dr;
  a.dz = dz;
  a.dw = dw;
  a.dw_post = dw_post;
  a.dscale = dscale;
  a.part = static_cast<float*>(workspace);
  return gdn::launch_residual_norm_backward(a, dtype, r_dtype, sms, st);
}

}  // extern "C"
