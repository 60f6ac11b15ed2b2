// Channel recurrence (gated linear recurrence) with a parallel scan over time,
// its single-token step and its backward pass.
//
//   forward   h_t   = alpha_t h_{t-1} + beta_t x_t,      alpha_t = exp(g_t)
//   backward  lam_t = dh_t + alpha_{t+1} lam_{t+1},      lam_T = dh_T + dstate
//             dx = beta lam, dbeta = x lam, dg = lam alpha_t h_{t-1},
//             dh_0 = alpha_1 lam_1
//
// Every channel is a chain of its own, so the work is a stream over memory (one
// exponential and a few multiply-adds an element): HBM bounds it.  Too few
// chains to fill the GPU one thread each, so time is cut as well.  Over a run of
// tokens the map from the state before it to the state behind it is affine,
// c -> exp(G) c + H, with G the sum of the run's log decays and H its end state
// from zero; the maps of neighbouring runs compose.
//
// A warp owns 32 V neighbouring channels of S consecutive tokens (a slice, held
// in registers), the W warps of a CTA own consecutive slices, and the CTAs of a
// cluster consecutive tiles of W S tokens; the cluster walks its sequence
// cluster-tile by cluster-tile.  Per cluster-tile each thread (1) takes its slice
// (from shared memory, where TMA has put it, or from registers that plain loads have
// filled), starts the fetch of the next one and finds its map, (2) leaves it in shared memory, where the CTA's map is composed
// and sent to the other CTAs of the cluster, (3) applies the maps before its own
// to the carried state and (4) walks its slice again from the right state,
// writing results.  Each element is read once and written once, no global memory
// carries partial results between CTAs, and the order of every sum is fixed:
// results do not depend on timing.
//
// States, maps and sums are fp32; bf16 is rounded to once, in a result.
//
// Measured (bf16 with beta, of the measured 6554 GB/s): forward 32768 x 4096 209 to 226
// us (91 to 98%), 4 x 4096 x 2048 59 us (89%); backward of the latter 111 us (84%).  The
// way there, on 32768 x 4096 forward: 1282 us with joins of exp(sum) at every step
// and predicated loads, 344 with small CTAs, one product a join and whole slices,
// 303 with the next slice prefetched, 283 with maps sent by st.async instead of
// cluster barriers, 207 to 216 with TMA instead of per-thread copies, and up to 10 us of
// that for decays and states at the ends of the fp32 range.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "gdn_host.h"
#include "gdn_internal.h"
#include "gdn_vec.cuh"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kCarryTokens = GDN_SCAN_CARRY_TOKENS;
constexpr int kMaxCluster = 8;  // CTAs along time
constexpr uint64_t kWaitLimitNs = 2000000000;  // 2 s: far beyond any legitimate wait
constexpr int kMaxSorted = 128;  // packed sequences that are started longest first

// The map of a run of tokens for V channels: c -> A c + H.  Where the run's growth
// passes the fp32 range A is infinite and so is what comes of a state, unless that is
// zero, which stays out of it.
template <int V>
struct alignas(8 * V) Map {
  F<V> A, H;
};
template <int V>
__device__ __forceinline__ F<V> apply(const Map<V>& m, F<V> c) {
  F<V> a = m.A;
#pragma unroll
  for (int e = 0; e < V; ++e) a.v[e] = c.v[e] == 0.f ? 0.f : a.v[e];
  return fma(a, c, m.H);
}
// The factor of run x before run y; a decay to nothing in one of them outweighs any
// growth in the other.
template <int V>
__device__ __forceinline__ F<V> join(F<V> x, F<V> y) {
  F<V> a = mul(x, y);
#pragma unroll
  for (int e = 0; e < V; ++e) a.v[e] = x.v[e] == 0.f || y.v[e] == 0.f ? 0.f : a.v[e];
  return a;
}

// A token's decay, exp(g) as 2^(g log2 e), the power by the approximate instruction
// (two units in the last place), below the normal numbers too, as a single token's
// expf.  (Three instructions more than with ftz, which makes those results zero: 32768 x
// 4096 forward 224 us against 220, 4096 x 2048 21.8 against 20.0; expf for every token
// 23.8 there; a branch around slices without such decays 266 by its registers.)
template <int V>
__device__ __forceinline__ F<V> decay(F<V> g) {
  g = mul(g, all<V>(1.4426950408889634f));
#pragma unroll
  for (int e = 0; e < V; ++e) asm("ex2.approx.f32 %0, %1;" : "=f"(g.v[e]) : "f"(g.v[e]));
  return g;
}
// A run's, from the sum of its log decays.
template <int V>
__device__ __forceinline__ F<V> run_decay(F<V> g) {
#pragma unroll
  for (int e = 0; e < V; ++e) g.v[e] = expf(g.v[e]);
  return g;
}

__device__ __forceinline__ unsigned cluster_size() {
  unsigned n;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Stores a map to the same shared-memory address in CTA `rank` of the cluster,
// counted by that CTA's mbarrier.
template <int V>
__device__ __forceinline__ void store_remote(Map<V>* local, uint64_t* bar, unsigned rank,
                                             const Map<V>& m) {
  unsigned a, b;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(a)
               : "r"(smem_u32(local)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(b)
               : "r"(smem_u32(bar)), "r"(rank));
  if constexpr (V == 2)
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%2, %3, %4, %5}, "
        "[%1];" ::"r"(a),
        "r"(b), "f"(m.A.v[0]), "f"(m.A.v[1]), "f"(m.H.v[0]), "f"(m.H.v[1])
        : "memory");
  else
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%2, %3}, [%1];" ::"r"(
            a),
        "r"(b), "f"(m.A.v[0]), "f"(m.H.v[0])
        : "memory");
}
struct Seq {
  long long start;  // first token
  int len;
  long long carry_row;
};

// The sequence `n` of the call; false if its packed offsets are invalid.
__device__ __forceinline__ bool sequence(const ScanArgs& a, int n, Seq* s) {
  if (!a.cu_seqlens) {
    s->start = (long long)n * a.T;
    s->len = a.T;
    s->carry_row = (long long)n * ((a.T + kCarryTokens - 1) / kCarryTokens);
    return true;
  }
  const int b = a.cu_seqlens[n], e = a.cu_seqlens[n + 1];
  if (b < 0 || e < b || e > a.T) return false;
  s->start = b;
  s->len = e - b;
  s->carry_row = b / kCarryTokens + n;
  return true;
}

// The sequence that CTA group r works on: with more CTAs than are resident, packed
// sequences start longest first (ties in order), so that a long one does not run
// alone at the end.  The same answer in every thread of every CTA of r.
__device__ __forceinline__ int pick_sequence(const ScanArgs& a, int r) {
  if (!a.sorted) return r;
  __shared__ int len[kMaxSorted], found;
  const int t = threadIdx.x;  // of kMaxSorted or more
  const int mine = t < a.N ? a.cu_seqlens[t + 1] - a.cu_seqlens[t] : 0;
  if (t < a.N) len[t] = mine;
  __syncthreads();
  int rank = 0;
  for (int j = 0; j < a.N; ++j) rank += len[j] > mine || (len[j] == mine && j < t);
  if (t < a.N && rank == r) found = t;
  __syncthreads();
  return found;
}

// Shared memory of the exchange: two sets, used in turn.  A set is written again
// only behind the wait for the other one, which every thread that reads it has
// passed by then (in this CTA by __syncthreads, in the cluster because a CTA
// sends the next tile's map only after that barrier).
template <int V, int W>
struct alignas(128) Exchange {
  uint64_t bar[2];                 // the cluster's maps of a set have arrived
  uint64_t full[W];                // a warp's slice has arrived (TMA)
  Map<V> warp[2][W][32];           // this CTA's slices, in scan order
  Map<V> cta[2][W >= 4 ? kMaxCluster : 1][32];  // the cluster's tiles, in scan order
};

// Before the first exchange and the first TMA.
template <int V, int W>
__device__ __forceinline__ void exchange_init(Exchange<V, W>& ex, unsigned n, bool tma) {
  if (n == 1 && !tma) return;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&ex.bar[0]), 1);
    mbar_init(smem_u32(&ex.bar[1]), 1);
#pragma unroll
    for (int i = 0; i < W; ++i) mbar_init(smem_u32(&ex.full[i]), 1);
    fence_mbar_init();
  }
  if (n > 1)
    cluster_barrier();  // every CTA runs, its barriers ready, before it is written to
  else
    __syncthreads();
}

// Shares the map of this thread's slice (scan order: CTA `rank`, warp `w`) and
// turns carry, the state before the cluster-tile, into the state before the
// slice (returned in c) and the state behind the cluster-tile (carry).  `round`
// counts the cluster-tiles.  Maps travel by st.async, counted by the receiver's
// mbarrier: a cluster barrier's release would wait for all of the CTA's stores
// to global memory as well.  The wait is bounded; a CTA that gave up once
// (*late) waits no more, goes on with what it has and reports it at the end.
template <int V, int W>
__device__ __forceinline__ void scan_exchange(Exchange<V, W>& ex, int round, const Map<V>& mine,
                                              F<V>& carry, F<V>& c, int w, int lane,
                                              unsigned rank, unsigned n, bool* late) {
  const int set = round & 1;
  ex.warp[set][w][lane] = mine;
  if (n > 1 && threadIdx.x == 0 && !*late)
    mbar_arrive_expect_tx(smem_u32(&ex.bar[set]), n * 32 * sizeof(Map<V>));
  __syncthreads();
  c = carry;
  if (n > 1) {
    if (w < n) {  // warp w composes the CTA's map for the CTAs w, w + W, ...
      Map<V> m = ex.warp[set][0][lane];
#pragma unroll
      for (int i = 1; i < W; ++i) {
        const Map<V> y = ex.warp[set][i][lane];
        m.H = apply(y, m.H);
        m.A = join(m.A, y.A);
      }
      for (unsigned r = w; r < n; r += W)
        store_remote(&ex.cta[set][rank][lane], &ex.bar[set], r, m);
    }
    mbar_wait_warp(smem_u32(&ex.bar[set]), (round >> 1) & 1, late, kWaitLimitNs);
    for (unsigned r = 0; r < n; ++r) {
      if (r == rank) c = carry;
      carry = apply(ex.cta[set][r][lane], carry);
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
      if (i < w) c = apply(ex.warp[set][i][lane], c);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (i == w) c = carry;
      carry = apply(ex.warp[set][i][lane], carry);
    }
  }
}

// Behind the last exchange: no CTA ends while another may still write to it.
// A warp whose wait ran out waits once more for the slice it has in flight.
__device__ __forceinline__ void exchange_end(unsigned n, bool late, int* status, uint64_t* full,
                                             unsigned issued) {
  if (late) {
    if (status) *status = GDN_ERR_DEVICE_TIMEOUT;
    bool again = false;
    if (issued > 0) mbar_wait_warp(smem_u32(full), (issued - 1) & 1, &again, kWaitLimitNs);
  }
  if (n > 1) cluster_barrier();
}

// How a slice gets from memory to registers, one slice ahead of the work on it.
// Two channels a thread (V = 2): by TMA, one lane a warp fetching the warp's
// slice, S tokens x 64 channels; a warp reads only what it fetched, so no barrier
// is needed.  One channel a thread, where TMA cannot go: by loads into registers.
// (Copies by cp.async, each thread its own elements, were slower than either:
// 32768 x 4096 forward 283 us against 207 by TMA; 5 x 577 x 577 in fp32 28 us
// against 10 by loads; loads of pairs, whose registers leave no room for the next
// slice, 16 x 1024 x 2050 95 us against 74.)

// A tile's slices: the log decays and K arrays of T.
template <typename T, int V, int S, int W, int K>
struct alignas(128) Stage {
  Vec<float, V> g[W][S][32];
  Vec<T, V> t[K][W][S][32];
};
struct ScanMaps {
  CUtensorMap g, t[3];
};

// TMA box of the map at (channel c, token row), counted by bar.
__device__ __forceinline__ void tma_rows(void* dst, const CUtensorMap* map, uint64_t* bar, int c,
                                         int row) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(bar)), "r"(c), "r"(row)
      : "memory");
}

// The slice's elements from the stage (tokens >= cnt of a TMA box are another
// sequence's: zeros instead).
template <typename E, int S>
__device__ __forceinline__ void take(E (&r)[S], const E (&src)[S][32], int cnt) {
#pragma unroll
  for (int i = 0; i < S; ++i) r[i] = src[i][threadIdx.x & 31];
  if (cnt < S) {
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (i >= cnt) r[i] = E{};
  }
}
// Starts loading them: tokens 0 .. cnt - 1 at p, zeros behind them.
template <typename E, int S>
__device__ __forceinline__ void load_slice(E (&r)[S], const void* p, size_t stride, int cnt) {
  const char* q = static_cast<const char*>(p);
#pragma unroll
  for (int i = 0; i < S; ++i) {
    r[i] = E{};
    if (i < cnt) r[i] = *reinterpret_cast<const E*>(q + i * stride);
  }
}
template <typename E, int S>
__device__ __forceinline__ void copy(E (&r)[S], const E (&x)[S]) {
#pragma unroll
  for (int i = 0; i < S; ++i) r[i] = x[i];
}

template <typename T, int V, int S, int W, bool BETA>
__global__ void __launch_bounds__(32 * W, 16 / W)
    scan_kernel(const ScanArgs a, const __grid_constant__ ScanMaps maps) {
  constexpr bool TMA = V == 2;
  extern __shared__ __align__(128) unsigned char smem[];
  auto& ex = *reinterpret_cast<Exchange<V, W>*>(smem);
  auto& st = *reinterpret_cast<Stage<T, V, S, W, BETA ? 2 : 1>*>(smem + sizeof(Exchange<V, W>));
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const unsigned n = cluster_size(), rank = cluster_rank();
  const int id = blockIdx.x / n, seq = pick_sequence(a, id / a.cblocks);
  int c0 = (id % a.cblocks) * 32 * V + lane * V;
  const bool on = c0 < a.C;
  if (!on) c0 = a.C - V;  // lanes past the last channel repeat it and store nothing
  Seq s;
  if (!sequence(a, seq, &s)) {  // the same answer in every CTA of the cluster
    if (a.status && threadIdx.x == 0 && rank == 0) *a.status = GDN_ERR_SHAPE;
    return;
  }
  F<V> carry{};  // (read ahead of the barrier: h_T may be h0, and one CTA writes it)
  if (a.h0) carry = to_f(load<float, V>(a.h0 + (size_t)seq * a.C + c0));
  exchange_init(ex, n, TMA);
  constexpr int tile = W * S;
  const int step = tile * int(n);
  [[maybe_unused]] const size_t gs = size_t(a.C) * 4, ts = size_t(a.C) * sizeof(T);
  int t0 = int(rank) * tile + w * S, cnt = 0;
  bool late = false;    // a wait ran out: nothing more is fetched or awaited
  unsigned issued = 0;  // slices fetched by TMA
  Vec<float, V> gn[TMA ? 1 : S];  // the next slice, on its way
  Vec<T, V> xn[TMA ? 1 : S], bn[TMA || !BETA ? 1 : S];
  // fetches the slice at token t0: tokens past the end are g = x = 0, which leaves
  // the state as it is; cnt is the same in every lane
  const auto place = [&] {
    cnt = min(max(s.len - t0, 0), S);
    if constexpr (TMA) {
      if (cnt > 0 && !late) {
        ++issued;
        if (lane == 0) {
          const int c = (id % a.cblocks) * 32 * V, row = int(s.start) + t0;
          mbar_arrive_expect_tx(smem_u32(&ex.full[w]),
                                sizeof(st.g[w]) + (BETA ? 2 : 1) * sizeof(st.t[0][w]));
          tma_rows(&st.g[w], &maps.g, &ex.full[w], c, row);
          tma_rows(&st.t[0][w], &maps.t[0], &ex.full[w], c, row);
          if (BETA) tma_rows(&st.t[BETA ? 1 : 0][w], &maps.t[1], &ex.full[w], c, row);
        }
      }
    } else {
      const size_t at = cnt > 0 ? size_t(s.start + t0) * a.C + c0 : 0;
      load_slice(gn, a.g + at, gs, cnt);
      load_slice(xn, static_cast<const T*>(a.x) + at, ts, cnt);
      if constexpr (BETA) load_slice(bn, static_cast<const T*>(a.beta) + at, ts, cnt);
    }
  };
  if (s.len > 0) place();
  int round = 0;
  for (int base = 0; base < s.len; base += step, ++round) {
    Vec<float, V> g[S];
    Vec<T, V> x[S], b[BETA ? S : 1];
    if constexpr (TMA) {
      if (cnt > 0) mbar_wait_warp(smem_u32(&ex.full[w]), (issued - 1) & 1, &late, kWaitLimitNs);
      take(g, st.g[w], cnt);
      take(x, st.t[0][w], cnt);
      if constexpr (BETA) take(b, st.t[1][w], cnt);
      __syncwarp();  // the next fetch overwrites what every lane has taken
    } else {
      copy(g, gn);
      copy(x, xn);
      if constexpr (BETA) copy(b, bn);
    }
    const int now = t0, have = cnt;
    t0 += step;
    if (base + step < s.len) place();  // in flight while this slice is worked on
    F<V> al[S], u[S], h;
    Map<V> m{};
#pragma unroll
    for (int i = 0; i < S; ++i) {
      al[i] = decay(to_f(g[i]));
      u[i] = BETA ? mul(to_f(x[i]), to_f(b[BETA ? i : 0])) : to_f(x[i]);
      m.A = add(m.A, to_f(g[i]));
      m.H = fma(al[i], m.H, u[i]);
    }
    m.A = run_decay(m.A);
    scan_exchange(ex, round, m, carry, h, w, lane, rank, n, &late);
    if (have > 0 && on && a.carries && now % kCarryTokens == 0)
      store<float, V>(a.carries + size_t(s.carry_row + now / kCarryTokens) * a.C + c0, h.v);
    if (a.h && on) {
      T* ph = static_cast<T*>(a.h) + (have > 0 ? size_t(s.start + now) * a.C + c0 : 0);
      if (have == S) {
#pragma unroll
        for (int i = 0; i < S; ++i) {
          h = fma(al[i], h, u[i]);
          store<T, V>(ph + (size_t)i * a.C, h.v);
        }
      } else {
#pragma unroll
        for (int i = 0; i < S; ++i) {
          h = fma(al[i], h, u[i]);
          if (i < have) store<T, V>(ph + (size_t)i * a.C, h.v);
        }
      }
    }
  }
  if (a.h_T && rank == 0 && w == 0 && on)
    store<float, V>(a.h_T + (size_t)seq * a.C + c0, carry.v);
  exchange_end(n, late, a.status, &ex.full[w], issued);
}

// Gradients of packed tokens that are before the first sequence or behind the last are
// zero: the CTAs of a channel block (group `r` of N, CTA `rank` of n in it) share them.
// Ends of invalid sequences leave everything as it was.
template <typename T, int V, int W>
__device__ __forceinline__ void zero_outside(const ScanBackwardArgs& a, int r, unsigned rank,
                                             unsigned n, int c0) {
  const ScanArgs& f = a.f;
  const int* cu = f.cu_seqlens;
  const int first = cu[0], last = cu[f.N];
  const int head = first >= 0 && first <= cu[1] && first <= f.T ? first : 0;
  const int tail = cu[f.N - 1] >= 0 && cu[f.N - 1] <= last && last <= f.T ? last : f.T;
  const long long rows = (long long)head + (f.T - tail), step = (long long)f.N * n * W;
  const float zero[V] = {};
  for (long long k = ((long long)r * n + rank) * W + (threadIdx.x >> 5); k < rows; k += step) {
    const size_t at = size_t(k < head ? k : tail + (k - head)) * f.C + c0;
    store<T, V>(static_cast<T*>(a.dx) + at, zero);
    store<float, V>(a.dg + at, zero);
    if (a.dbeta) store<T, V>(static_cast<T*>(a.dbeta) + at, zero);
  }
}

// Backward: the same walk from the sequence's end.  What passes a token
// boundary is mu_t = alpha_t lam_t.  h_{t-1} is rebuilt in 32 bits from the
// states that the forward pass kept every 16 tokens: reading them costs 4/16
// byte an element, reading h itself 2 to 4 and, in bf16, its rounding in dg.
template <typename T, int V, int S, int W, bool BETA>
__global__ void __launch_bounds__(32 * W, 16 / W)
    scan_backward_kernel(const ScanBackwardArgs a, const __grid_constant__ ScanMaps maps) {
  constexpr bool TMA = V == 2;
  // the later slices of a kept state's 16 tokens start from the slices before
  constexpr int M = kCarryTokens / S;
  extern __shared__ __align__(128) unsigned char smem[];
  auto& ex = *reinterpret_cast<Exchange<V, W>*>(smem);
  auto& fwd = *reinterpret_cast<Map<V>(*)[2][W][32]>(smem + sizeof(Exchange<V, W>));
  auto& st = *reinterpret_cast<Stage<T, V, S, W, BETA ? 3 : 2>*>(smem + sizeof(Exchange<V, W>) +
                                                              sizeof(fwd));
  const ScanArgs& f = a.f;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const unsigned n = cluster_size(), rank = cluster_rank();
  const int id = blockIdx.x / n, seq = pick_sequence(f, id / f.cblocks);
  int c0 = (id % f.cblocks) * 32 * V + lane * V;
  const bool on = c0 < f.C;
  if (!on) c0 = f.C - V;
  if (f.cu_seqlens && on) zero_outside<T, V, W>(a, id / f.cblocks, rank, n, c0);
  Seq s;
  if (!sequence(f, seq, &s)) {
    if (f.status && threadIdx.x == 0 && rank == 0) *f.status = GDN_ERR_SHAPE;
    return;
  }
  F<V> carry{};
  if (a.dh_T) carry = to_f(load<float, V>(a.dh_T + (size_t)seq * f.C + c0));
  exchange_init(ex, n, TMA);
  constexpr int tile = W * S;
  const int tiles = (s.len + tile - 1) / tile;
  const int sw = W - 1 - w;  // scan order runs backwards in time
  [[maybe_unused]] const size_t gs = size_t(f.C) * 4, ts = size_t(f.C) * sizeof(T);
  int ti = tiles - 1 - int(rank), cnt = 0;  // the tile; below 0: past the start
  size_t at = 0;
  Vec<float, V> kept{};
  bool late = false;
  unsigned issued = 0;
  Vec<float, V> gn[TMA ? 1 : S];
  Vec<T, V> dn[TMA ? 1 : S], xn[TMA ? 1 : S], bn[TMA || !BETA ? 1 : S];
  const auto place = [&] {
    const int t0 = ti * tile + sw * S;
    cnt = ti >= 0 ? min(max(s.len - t0, 0), S) : 0;
    at = cnt > 0 ? size_t(s.start + t0) * f.C + c0 : 0;
    if constexpr (TMA) {
      if (cnt > 0 && !late) {
        ++issued;
        if (lane == 0) {
          const int c = (id % f.cblocks) * 32 * V, row = int(s.start) + t0;
          mbar_arrive_expect_tx(smem_u32(&ex.full[w]),
                                sizeof(st.g[w]) + (BETA ? 3 : 2) * sizeof(st.t[0][w]));
          tma_rows(&st.g[w], &maps.g, &ex.full[w], c, row);
          tma_rows(&st.t[0][w], &maps.t[0], &ex.full[w], c, row);
          tma_rows(&st.t[1][w], &maps.t[1], &ex.full[w], c, row);
          if (BETA) tma_rows(&st.t[BETA ? 2 : 0][w], &maps.t[2], &ex.full[w], c, row);
        }
      }
    } else {
      load_slice(gn, f.g + at, gs, cnt);
      load_slice(dn, static_cast<const T*>(a.dh) + at, ts, cnt);
      load_slice(xn, static_cast<const T*>(f.x) + at, ts, cnt);
      if constexpr (BETA) load_slice(bn, static_cast<const T*>(f.beta) + at, ts, cnt);
    }
    if (cnt > 0)
      kept = load<float, V>(f.carries + size_t(s.carry_row + t0 / kCarryTokens) * f.C + c0);
  };
  if (tiles > 0) place();
  int round = 0;
  for (int first = 0; first < tiles; first += int(n), ++round) {
    const int set = round & 1;
    Vec<float, V> g[S];
    Vec<T, V> x[S], b[BETA ? S : 1], d[S];
    if constexpr (TMA) {
      if (cnt > 0) mbar_wait_warp(smem_u32(&ex.full[w]), (issued - 1) & 1, &late, kWaitLimitNs);
      take(g, st.g[w], cnt);
      take(d, st.t[0][w], cnt);
      take(x, st.t[1][w], cnt);
      if constexpr (BETA) take(b, st.t[2][w], cnt);
      __syncwarp();
    } else {
      copy(g, gn);
      copy(d, dn);
      copy(x, xn);
      if constexpr (BETA) copy(b, bn);
    }
    F<V> h = to_f(kept), mu;
    const size_t out = at;
    const int have = cnt;
    ti -= int(n);
    if (first + int(n) < tiles) place();
    const auto input = [&](int i) {
      return BETA ? mul(to_f(x[i]), to_f(b[BETA ? i : 0])) : to_f(x[i]);
    };
    F<V> al[S];
    Map<V> m{}, mf{};
#pragma unroll
    for (int i = 0; i < S; ++i) {
      al[i] = decay(to_f(g[i]));
      m.A = add(m.A, to_f(g[i]));
      if (M > 1) mf.H = fma(al[i], mf.H, input(i));
    }
#pragma unroll
    for (int i = S - 1; i >= 0; --i) m.H = mul(al[i], add(to_f(d[i]), m.H));
    mf.A = m.A = run_decay(m.A);
    if (M > 1) fwd[set][sw][lane] = mf;
    scan_exchange(ex, round, m, carry, mu, w, lane, rank, n, &late);
    if (M > 1) {
#pragma unroll
      for (int i = 0; i < M - 1; ++i)
        if (i < sw % M) h = apply(fwd[set][sw - sw % M + i][lane], h);
    }
    F<V> hp[S];  // h before each token
#pragma unroll
    for (int i = 0; i < S; ++i) {
      hp[i] = h;
      h = fma(al[i], h, input(i));
    }
#pragma unroll
    for (int i = S - 1; i >= 0; --i) {
      const F<V> lam = add(to_f(d[i]), mu);
      mu = mul(al[i], lam);
      if (on && i < have) {
        const size_t o = out + (size_t)i * f.C;
        store<T, V>(static_cast<T*>(a.dx) + o, (BETA ? mul(lam, to_f(b[BETA ? i : 0])) : lam).v);
        store<float, V>(a.dg + o, mul(mu, hp[i]).v);
        if (BETA) store<T, V>(static_cast<T*>(a.dbeta) + o, mul(lam, to_f(x[i])).v);
      }
    }
  }
  if (a.dh0 && rank == 0 && w == 0 && on)
    store<float, V>(a.dh0 + (size_t)seq * f.C + c0, carry.v);
  exchange_end(n, late, f.status, &ex.full[w], issued);
}

// One token: elementwise, V channels a thread.
template <typename T, int V, bool BETA>
__global__ void __launch_bounds__(256) scan_step_kernel(const T* x, const float* g, const T* beta,
                                                        float* state, T* h, size_t count) {
  const size_t i = (size_t(blockIdx.x) * 256 + threadIdx.x) * V;
  if (i >= count) return;
  const Vec<T, V> vx = load<T, V>(x + i);
  const Vec<float, V> vg = load<float, V>(g + i), vs = load<float, V>(state + i);
  Vec<T, V> vb;
  if (BETA) vb = load<T, V>(beta + i);
  float r[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float u = BETA ? to_f(vx.v[e]) * to_f(vb.v[e]) : to_f(vx.v[e]);
    r[e] = fmaf(expf(vg.v[e]), vs.v[e], u);
  }
  store<float, V>(state + i, r);
  store<T, V>(h + i, r);
}

// Warps of a CTA and CTAs of a cluster, both along time.  16 warps an SM are
// resident at 128 registers.  In microseconds, forward / backward, at bf16 with beta:
//   few     (one 16-token slice, or chains enough to fill the GPU one warp each)
//           64 x 16 x 4096: 12 / 19 against 24 / 27 on four warps
//           (equal lengths; a far longer sequence among many is walked by these warps
//           alone: one of 16384 tokens with 127 of 64, 2048 channels, 885 / 1167)
//   packed  sequences end at different times, so more CTAs are started than are
//           resident.  8 sequences, 8192 x 2048 (256 chains): 38 / 68 on clusters of
//           4, 45 / 96 on 2, 45 / 70 on 8; 64, 32768 x 512 (512 chains): 46 / 71, 45
//           / 93, 65 / 91.  32, 16384 x 2048 (1024 chains): 58 / 107 on one CTA of
//           eight warps, 64 / 112 on two of four, 80 / 129 on four
//   8, n=1  1.5 to 4 chains an SM: 8 x 2048 x 2048 56 / 111, four warps on two CTAs
//           59 / 126
//   4, n    else as many CTAs as are resident at once: 4 x 4096 x 2048 86 / 190 on
//           1, 62 / 137 on 2, 58 / 108 on 4, 62 / 112 on 8 (two waves)
//   8, n=8  so few chains that even this is resident: 4096 x 2048 20 / 35 against
//           21 / 42 on four warps
// A tenth of what is resident is left free: clusters do not fill every GPC.
struct Shape {
  int warps, cluster;
};
Shape pick_shape(const ScanArgs& a, int S, long long chains, int sms, int few) {
  const bool packed = a.cu_seqlens && a.N > 1;
  const long long len = a.cu_seqlens ? std::max<long long>(1, a.T / std::max(1, a.N)) : a.T;
  if (len <= few * S || chains >= 16LL * sms) return {few, 1};
  const auto resident = [&](int warps) { return 16 / warps * (long long)sms * 9 / 10; };
  int W = 4;
  if (len > 4 * S && (packed ? 4 * chains > 14LL * sms
                             : (2 * chains >= 3LL * sms && chains <= 4LL * sms) ||
                                   chains * kMaxCluster <= resident(8)))
    W = 8;
  int n = 1;
  if (packed)
    n = W == 8 ? 1 : 8 * chains <= 4LL * sms ? 8 : 4;
  else
    while (n < kMaxCluster && chains * n * 2 <= resident(W)) n *= 2;
  while (n > 1 && (n / 2) * (long long)W * S >= len) n /= 2;  // each CTA has tokens
  return {W, n};
}

// go(warps, has beta), both as types.
template <int FEW, typename Go>
bool dispatch_scan(int warps, bool beta, Go&& go) {
  const auto sized = [&](auto w) {
    return beta ? go(w, std::true_type{}) : go(w, std::false_type{});
  };
  if constexpr (FEW < 4)
    if (warps == FEW) return sized(std::integral_constant<int, FEW>{});
  if (warps == 8) return sized(std::integral_constant<int, 8>{});
  return sized(std::integral_constant<int, 4>{});
}

template <auto Kernel, typename Args>
bool launch_cluster(const Args& args, const ScanMaps& maps, int threads, size_t smem,
                    long long ctas, int n, cudaStream_t stream) {
  if (!raise_smem<Kernel>(smem)) return false;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(ctas * n));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = unsigned(n);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = n > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, Kernel, args, maps) == cudaSuccess;
}

// The shape of a launch, its channel blocks and the order of its sequences.
template <int V>
bool plan(ScanArgs& a, int S, int few, int sms, long long* chains, Shape* shape) {
  a.cblocks = (a.C + 32 * V - 1) / (32 * V);
  *chains = (long long)a.cblocks * a.N;
  if (*chains * kMaxCluster > 0x7fffffffLL) return false;
  *shape = pick_shape(a, S, *chains, sms, few);
  a.sorted = a.cu_seqlens && a.N <= kMaxSorted && shape->warps >= 4 &&
             *chains * shape->cluster > 16 / shape->warps * (long long)sms;
  return true;
}

template <typename T, int V, int S>
int run_scan(ScanArgs a, int sms, cudaStream_t stream) {
  constexpr int kFew = V == 2 ? 1 : 4;
  long long chains;
  Shape sh;
  if (!plan<V>(a, S, kFew, sms, &chains, &sh)) return GDN_ERR_SHAPE;
  const long long rows = a.cu_seqlens ? a.T : (long long)a.N * a.T;
  constexpr bool bf16 = sizeof(T) == 2;
  ScanMaps maps{};
  if (V == 2 && rows > 0 &&
      !(encode_rows(&maps.g, a.g, rows, a.C, 64, S, false) &&
        encode_rows(&maps.t[0], a.x, rows, a.C, 64, S, bf16) &&
        (!a.beta || encode_rows(&maps.t[1], a.beta, rows, a.C, 64, S, bf16))))
    return GDN_ERR_LAUNCH;
  const auto go = [&](auto warps, auto beta) {
    constexpr int W = decltype(warps)::value;
    constexpr bool kBeta = decltype(beta)::value;
    constexpr size_t smem =
        sizeof(Exchange<V, W>) + (V == 2 ? sizeof(Stage<T, V, S, W, kBeta ? 2 : 1>) : 0);
    return launch_cluster<&scan_kernel<T, V, S, W, kBeta>>(a, maps, 32 * W, smem, chains,
                                                           sh.cluster, stream);
  };
  return dispatch_scan<kFew>(sh.warps, a.beta != nullptr, go) ? GDN_OK : GDN_ERR_LAUNCH;
}

template <typename T, int V, int S>
int run_backward(ScanBackwardArgs a, int sms, cudaStream_t stream) {
  constexpr int kFew = V == 2 ? kCarryTokens / S : 4;
  static_assert(kFew * S % kCarryTokens == 0, "a tile starts at a kept state");
  ScanArgs& f = a.f;
  long long chains;
  Shape sh;
  if (!plan<V>(f, S, kFew, sms, &chains, &sh)) return GDN_ERR_SHAPE;
  const long long rows = f.cu_seqlens ? f.T : (long long)f.N * f.T;
  constexpr bool bf16 = sizeof(T) == 2;
  ScanMaps maps{};
  if (V == 2 && rows > 0 &&
      !(encode_rows(&maps.g, f.g, rows, f.C, 64, S, false) &&
        encode_rows(&maps.t[0], a.dh, rows, f.C, 64, S, bf16) &&
        encode_rows(&maps.t[1], f.x, rows, f.C, 64, S, bf16) &&
        (!f.beta || encode_rows(&maps.t[2], f.beta, rows, f.C, 64, S, bf16))))
    return GDN_ERR_LAUNCH;
  const auto go = [&](auto warps, auto beta) {
    constexpr int W = decltype(warps)::value;
    constexpr bool kBeta = decltype(beta)::value;
    constexpr size_t smem = sizeof(Exchange<V, W>) + sizeof(Map<V>[2][W][32]) +
                            (V == 2 ? sizeof(Stage<T, V, S, W, kBeta ? 3 : 2>) : 0);
    return launch_cluster<&scan_backward_kernel<T, V, S, W, kBeta>>(a, maps, 32 * W, smem, chains,
                                                                    sh.cluster, stream);
  };
  return dispatch_scan<kFew>(sh.warps, f.beta != nullptr, go) ? GDN_OK : GDN_ERR_LAUNCH;
}

// Two channels a thread and TMA: rows of 64 channels or more, inputs whose rows and
// bases are multiples of 16 bytes, outputs and states that start on a pair.
// Encoding the maps takes the host some tenths of a microsecond (16 x 2048: 5.4 us
// a call against 5.2 with loads, 128 x 2048: 6.4 against 6.5, backward 6.2 against
// 6.1 and 6.5 against 7.0).
bool wide_ok(int C, int esize, std::initializer_list<const void*> in,
             std::initializer_list<const void*> out, std::initializer_list<const void*> f32) {
  if (C < 64 || C * (long long)esize % 16 != 0) return false;
  const auto all = [](std::initializer_list<const void*> v, uintptr_t n) {
    return std::all_of(v.begin(), v.end(), [n](const void* p) { return aligned(p, n); });
  };
  return all(in, 16) && all(out, 2 * uintptr_t(esize)) && all(f32, 8);
}

}  // namespace

int launch_scan(const ScanArgs& a, int dtype, int sms, cudaStream_t stream) {
  const int e = dtype == GDN_BF16 ? 2 : 4;
  const bool wide = wide_ok(a.C, e, {a.x, a.g, a.beta}, {a.h}, {a.h0, a.h_T, a.carries});
  if (dtype == GDN_BF16)
    return wide ? run_scan<__nv_bfloat16, 2, 16>(a, sms, stream)
                : run_scan<__nv_bfloat16, 1, 16>(a, sms, stream);
  return wide ? run_scan<float, 2, 8>(a, sms, stream) : run_scan<float, 1, 16>(a, sms, stream);
}

int launch_scan_backward(const ScanBackwardArgs& a, int dtype, int sms, cudaStream_t stream) {
  const int e = dtype == GDN_BF16 ? 2 : 4;
  const bool wide = wide_ok(a.f.C, e, {a.f.x, a.f.g, a.f.beta, a.dh}, {a.dx, a.dbeta},
                            {a.dg, a.dh_T, a.dh0, a.f.carries});
  if (dtype == GDN_BF16)
    return wide ? run_backward<__nv_bfloat16, 2, 8>(a, sms, stream)
                : run_backward<__nv_bfloat16, 1, 8>(a, sms, stream);
  return wide ? run_backward<float, 2, 8>(a, sms, stream)
              : run_backward<float, 1, 8>(a, sms, stream);
}

template <typename T, int V>
static int run_step(const ScanArgs& a, size_t count, cudaStream_t stream) {
  const unsigned grid = unsigned((count / V + 255) / 256);
  const T *x = static_cast<const T*>(a.x), *b = static_cast<const T*>(a.beta);
  if (a.beta)
    scan_step_kernel<T, V, true><<<grid, 256, 0, stream>>>(x, a.g, b, a.h_T, static_cast<T*>(a.h),
                                                           count);
  else
    scan_step_kernel<T, V, false><<<grid, 256, 0, stream>>>(x, a.g, b, a.h_T, static_cast<T*>(a.h),
                                                            count);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

int launch_scan_step(const ScanArgs& a, int dtype, cudaStream_t stream) {
  const size_t count = size_t(a.N) * a.C;
  const auto ok = [](const void* p, uintptr_t m) {
    return (reinterpret_cast<uintptr_t>(p) & (m - 1)) == 0;
  };
  const uintptr_t e4 = dtype == GDN_BF16 ? 8 : 16;
  const bool quads = count % 4 == 0 && ok(a.x, e4) && ok(a.beta, e4) && ok(a.h, e4) &&
                     ok(a.g, 16) && ok(a.h_T, 16);
  if (dtype == GDN_BF16)
    return quads ? run_step<__nv_bfloat16, 4>(a, count, stream)
                 : run_step<__nv_bfloat16, 1>(a, count, stream);
  return quads ? run_step<float, 4>(a, count, stream) : run_step<float, 1>(a, count, stream);
}

}  // namespace gdn
