// C-ABI entry points of the channel recurrence: argument checks, then the
// launches on the caller's stream.
#include <algorithm>

#include "gdn_host.h"
#include "gdn_internal.h"

namespace {

using gdn::aligned;
using gdn::Span;

constexpr long long kMaxTokens = 1LL << 30;
constexpr long long kMaxElements = 1LL << 40;

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

}  // namespace

extern "C" {

size_t gdn_scan_carry_bytes(int N, int tokens, int C, int packed) {
  if (N < 0 || tokens < 0 || C < 0) return 0;
  return size_t(carry_rows(N, tokens, packed != 0)) * size_t(C) * 4;
}

int gdn_scan(const void* x, const float* g, const void* beta, const float* h0, void* h, float* h_T,
             float* carries, int B, int T, int C, int dtype, void* stream) {
  if (B < 0 || T < 0) return GDN_ERR_SHAPE;
  return scan_impl({x, g, beta, h0, h, h_T, carries, nullptr, B, T, C, 0, nullptr},
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
                      int dtype, void* stream) {
  if (B < 0 || T < 0) return GDN_ERR_SHAPE;
  return scan_backward_impl(
      {{x, g, beta, h0, nullptr, nullptr, carries, nullptr, B, T, C, 0, nullptr}, dh, dh_T, dx, dg,
       dbeta, dh0},
      carries_valid, (long long)B * T, dtype, stream);
}

int gdn_scan_varlen_backward(const void* x, const float* g, const void* beta, const float* h0,
                             const void* dh, const float* dh_T, void* dx, float* dg, void* dbeta,
                             float* dh0, float* carries, int carries_valid, const int* cu_seqlens,
                             int N, int total_T, int C, int dtype, int* status, void* stream) {
  if (N > 0 && C > 0 && total_T >= 0 && !cu_seqlens) return GDN_ERR_NULL;
  return scan_backward_impl(
      {{x, g, beta, h0, nullptr, nullptr, carries, cu_seqlens, N, total_T, C, 0, status}, dh, dh_T,
       dx, dg, dbeta, dh0},
      carries_valid, total_T, dtype, stream);
}

}  // extern "C"
