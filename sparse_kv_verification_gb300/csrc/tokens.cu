// Verification of drafted tokens against the target's probabilities
// (speculative sampling): accept the longest run of drafts with
// u_i q_i(x_i) < p_i(x_i), then draw one token from the residual
// max(p - q, 0) at the first rejection, or from the target's next row.
//
// One cluster of C CTAs per sequence (C by the number of sequences, so that
// small batches still spread a vocabulary row over many SMs).
//  * Every CTA decides the accepted count on its own (one warp, 32 drafts at
//    a time, a ballot): 4 loads per draft, cheaper than telling the others.
//    The products u q are formed in fp64, where two fp32 factors are exact.
//  * The row's masses are summed once: CTA, warp and lane own nested
//    contiguous ranges.  A token's place in a 152k-entry running sum turns on
//    differences far below an fp32 ulp of the total, and fp64 arithmetic runs
//    at 1/64 of the fp32 rate here, so lanes sum in float-float: p - q and
//    each addition carry their exact rounding error along (TwoSum, about 48
//    bits); warp, CTA and cluster sums are fp64, added in rank order, so the
//    result does not depend on timing.
//  * The CTA whose range holds u * total walks it again (one warp's share,
//    1/(16 C) of the row, from L2) with a block scan of the same sums.
// One launch, no workspace, no atomics on device memory but the error flag's
// (the walk's maximum and minimum of entry numbers are shared memory's, and do
// not depend on their order).
//
// Bound by latency: the chain launch, draft's probabilities, row, cluster
// barrier, second walk.  Measured (one call after the other): 16 rows of
// 152064 in fp32, drafts rejected at random, 13.7 us (its 19.4 MB alone take
// 2.9), 64 rows of 50257 in bf16 at odd alignments 13.8, one row of 32000
// 7.9.  (Read element by element, the odd rows took 20.9.)
#include <algorithm>
#include <cooperative_groups.h>

#include "device_common.cuh"
#include "dustin.h"
#include "internal.h"

namespace cg = cooperative_groups;

namespace dustin {

namespace {

__device__ unsigned int g_tokens_dev_flags;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

// An unevaluated sum s + c, c within rounding of s.
struct Ff {
  float s, c;
};
__device__ __forceinline__ Ff two_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Ff ff_add(Ff x, Ff y) {
  const Ff t = two_sum(x.s, y.s);
  return {t.s, __fadd_rn(t.c, __fadd_rn(x.c, y.c))};
}
__device__ __forceinline__ double ff_value(Ff x) { return (double)x.s + (double)x.c; }

// A probability that counts: positive and finite (NaN, infinities and
// negative entries have no mass).
__device__ __forceinline__ float mass_of(float x) {
  return x > 0.f && x <= 3.402823466e38f ? x : 0.f;
}
// max(p - q, 0) as an exact float-float.
__device__ __forceinline__ Ff rest_of(float p, float q) {
  const float a = mass_of(p), b = mass_of(q);
  return a > b ? two_sum(a, -b) : Ff{0.f, 0.f};
}

template <typename T>
__device__ __forceinline__ float load1(const T* p) {
  if constexpr (sizeof(T) == 4)
    return __ldg(reinterpret_cast<const float*>(p));
  else
    return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p)) << 16);
}

__device__ __forceinline__ uint4 load16(const void* p) {
  return __ldg(reinterpret_cast<const uint4*>(p));
}
// 16 bytes as floats.
template <typename T>
__device__ __forceinline__ void to_floats(const uint4& u, float (&x)[16 / sizeof(T)]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = __uint_as_float(w[i]);
    } else {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// One sequence's row: target, and what is taken off it.
template <typename T>
struct Row {
  const T* p;
  const T* q;     // null: nothing, but entry `gone` has no mass
  long long gone; // -1: every entry counts
  __device__ __forceinline__ Ff at(long long j) const {
    const float pv = load1(p + j);
    if (q) return rest_of(pv, load1(q + j));
    return {j == gone ? 0.f : mass_of(pv), 0.f};
  }
};

// 16 bytes from byte `at` of the 32 in w (at: 0 .. 15, a multiple of the
// element size, the same for the whole warp): words, then a half word.
template <typename T>
__device__ __forceinline__ uint4 extract16(const uint4& lo, const uint4& hi, int at) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (at & 8)
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  if (at & 4)
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  if (sizeof(T) == 2 && (at & 2))
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __byte_perm(w[i], w[i + 1], 0x5432);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The calling lane's share of the mass in [lo, hi), float-float.  Rows start
// at any element: 16-byte loads follow p's alignment, and q's bytes, aligned
// otherwise, are put together from two of its 16-byte words (the second one
// the next lane's first).
template <typename T>
__device__ Ff lane_mass(const Row<T>& r, long long lo, long long hi, int lane) {
  constexpr int V = 16 / sizeof(T);
  Ff acc{0.f, 0.f};
  const int head = (int)((16 - (reinterpret_cast<uintptr_t>(r.p + lo) & 15u)) & 15u) / (int)sizeof(T);
  const long long j0 = min(hi, lo + head);
  if (lo + lane < j0) acc = ff_add(acc, r.at(lo + lane));
  const long long full = j0 + (hi - j0) / (32 * V) * (32 * V);
  if (!r.q) {
#pragma unroll 4
    for (long long j = j0; j < full; j += 32 * V) {
      const long long e = j + lane * V;
      float pv[V];
      to_floats<T>(load16(r.p + e), pv);
#pragma unroll
      for (int i = 0; i < V; ++i) acc = ff_add(acc, Ff{e + i == r.gone ? 0.f : mass_of(pv[i]), 0.f});
    }
  } else {
    const int off = (int)(reinterpret_cast<uintptr_t>(r.q + j0) & 15u);
#pragma unroll 2
    for (long long j = j0; j < full; j += 32 * V) {
      const long long e = j + lane * V;
      const uint4 pw = load16(r.p + e);
      const char* qa = reinterpret_cast<const char*>(r.q + e) - off;
      uint4 qw = load16(qa);
      if (off) {   // uniform
        uint4 next;
        next.x = __shfl_down_sync(0xffffffffu, qw.x, 1);
        next.y = __shfl_down_sync(0xffffffffu, qw.y, 1);
        next.z = __shfl_down_sync(0xffffffffu, qw.z, 1);
        next.w = __shfl_down_sync(0xffffffffu, qw.w, 1);
        // The last lane's second word holds an element of this range, too.
        if (lane == 31) next = load16(qa + 16);
        qw = extract16<T>(qw, next, off);
      }
      float pv[V], qv[V];
      to_floats<T>(pw, pv);
      to_floats<T>(qw, qv);
#pragma unroll
      for (int i = 0; i < V; ++i) acc = ff_add(acc, rest_of(pv[i], qv[i]));
    }
  }
  for (long long j = full + lane; j < hi; j += 32) acc = ff_add(acc, r.at(j));
  return acc;
}

// Inclusive sums over 16 lanes (both halves of the warp alike), in lane order.
__device__ __forceinline__ double scan16(double x, int lane) {
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, d, 16);
    if ((lane & 15) >= d) x += y;
  }
  return x;
}

struct Shared {
  double warp_sum[kWarps];
  double warp_base[kWarps + 1];   // sums below each warp, in the final walk
  double cta_sum;                 // read by the other CTAs of the cluster
  double total, base, t;
  int accepted;
  int walk;                       // warp range to walk (-1: another CTA's)
  int last;                       // last positive entry that starts at or below t
  int found;
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) verify_tokens_kernel(const TokenArgs a) {
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int bb = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();
  griddep_launch_dependents();

  // Read early: it is needed at the end of a chain of loads.
  const float u_here = warp == 0 ? __ldg(a.u_sample + bb) : 0.f;
  const T* p0 = static_cast<const T*>(a.p) + (long long)bb * a.stride_tb;
  const T* q0 = a.q ? static_cast<const T*>(a.q) + (long long)bb * a.stride_db : nullptr;
  const int* draft = a.draft ? a.draft + (long long)bb * (a.w - 1) : nullptr;
  int drafts = a.w - 1;
  if (a.n_draft) drafts = min(max(__ldg(a.n_draft + bb), 0), drafts);

  if (warp == 0) {
    int acc = 0;
    for (int base = 0; base < drafts; base += 32) {
      const int i = base + lane;
      bool ok = false;
      if (i < drafts) {
        const int x = __ldg(draft + i);
        if (x >= 0 && x < a.vocab) {
          const double u = (double)__ldg(a.u_accept + (long long)bb * (a.w - 1) + i);
          const double pv = (double)mass_of(load1(p0 + (long long)i * a.stride_tw + x));
          const double qv = q0 ? (double)mass_of(load1(q0 + (long long)i * a.stride_dw + x)) : 1.0;
          ok = u * qv < pv;
        } else if (rank == 0) {
          atomicOr(&g_tokens_dev_flags, DUSTIN_DEVFLAG_INDEX_RANGE);
        }
      }
      const unsigned no = __ballot_sync(0xffffffffu, !ok);
      if (no) {
        acc = base + __ffs((int)no) - 1;
        break;
      }
      acc = base + 32;
    }
    if (lane == 0) sh.accepted = min(acc, drafts);
  }
  __syncthreads();
  const int n_acc = sh.accepted;
  const bool rejected = n_acc < drafts;
  if (rank == 0) {
    for (int i = tid; i < a.w; i += kThreads)
      if (i != n_acc) a.tokens[(long long)bb * a.w + i] = i < n_acc ? __ldg(draft + i) : -1;
    if (tid == 0) a.n_accepted[bb] = n_acc;
  }

  // Nested ranges, each a multiple of 8 entries (16 bytes in either type).
  const long long per_warp = (((long long)a.vocab + C * kWarps - 1) / (C * kWarps) + 7) / 8 * 8;
  const long long lo = min((long long)a.vocab, (rank * kWarps + warp) * per_warp);
  const long long hi = min((long long)a.vocab, lo + per_warp);

  Row<T> row;
  row.p = p0 + (long long)n_acc * a.stride_tw;
  row.q = rejected && q0 ? q0 + (long long)n_acc * a.stride_dw : nullptr;
  row.gone = rejected && !q0 ? (long long)__ldg(draft + n_acc) : -1;
  // fp64 sums below run in one warp: an fp64 addition holds the unit for 16
  // cycles, whoever needs the result.
  for (int pass = 0; pass < 2; ++pass) {
    Ff acc = lane_mass(row, lo, hi, lane);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      acc = ff_add(acc, Ff{__shfl_xor_sync(0xffffffffu, acc.s, d),
                           __shfl_xor_sync(0xffffffffu, acc.c, d)});
    if (lane == 0) sh.warp_sum[warp] = ff_value(acc);
    __syncthreads();
    // Warp 0: inclusive sums over the CTA's warps, then over the CTAs.
    double mine = 0.0, run = 0.0;
    if (warp == 0) {
      mine = lane < kWarps ? sh.warp_sum[lane] : 0.0;
      run = scan16(mine, lane);
      if (lane == kWarps - 1) sh.cta_sum = run;
    }
    cl.sync();
    if (warp == 0) {
      const double theirs = lane < C ? *cl.map_shared_rank(&sh.cta_sum, lane) : 0.0;
      const double upto = scan16(theirs, lane);
      const double total = __shfl_sync(0xffffffffu, upto, kWarps - 1);
      const double before = rank ? __shfl_sync(0xffffffffu, upto, rank - 1) : 0.0;
      // From u = 1 on, the last token with mass, however little: its mass need
      // not show in the sums, so no finite t finds it.
      const bool top = u_here >= 1.f;
      const double t = top ? (double)INFINITY : u_here > 0.f ? (double)u_here * total : 0.0;
      // The first range with mass that ends behind t, the last one with mass
      // should rounding at the upper end leave none.
      // A range starts where the one below ends, and never beyond t: the walk
      // would find every sum past t at once.
      const double below = __shfl_up_sync(0xffffffffu, run, 1);
      const double base = fmin(lane ? before + below : before, t);
      const unsigned has = __ballot_sync(0xffffffffu, mine > 0.0);
      const unsigned ends = __ballot_sync(0xffffffffu, mine > 0.0 && before + run > t);
      const double after = __shfl_sync(0xffffffffu, upto, rank);
      const unsigned ctas = __ballot_sync(0xffffffffu, theirs > 0.0);
      const bool owner = top ? ctas && 31 - __clz((int)ctas) == rank
                             : total > 0.0 && before <= t && t < after && has;
      const int walk = owner ? (ends ? __ffs((int)ends) - 1 : 31 - __clz((int)has)) : -1;
      const double at = __shfl_sync(0xffffffffu, base, walk < 0 ? 0 : walk);
      if (lane == 0) {
        sh.total = total;
        sh.t = t;
        sh.base = at;
        sh.walk = walk;
        sh.last = -1;
        sh.found = 0x7fffffff;
      }
    }
    __syncthreads();
    // An empty residual (the draft's row covers the target's): the target's
    // row itself.  The same in every CTA of the cluster.
    if (sh.total > 0.0 || !rejected || pass) break;
    row.q = nullptr;
    row.gone = -1;
    cl.sync();   // cta_sum is read before the second pass writes it
  }

  if (sh.walk >= 0) {
    const double t = sh.t;
    const long long wlo = min((long long)a.vocab, (rank * kWarps + sh.walk) * per_warp);
    const long long whi = min((long long)a.vocab, wlo + per_warp);
    constexpr int E = 4;   // consecutive entries of a thread
    for (long long c0 = wlo; c0 < whi; c0 += kThreads * E) {
      Ff x[E];
      Ff mine{0.f, 0.f};
      int with_mass = -1;   // the thread's last such entry
      const long long j0 = c0 + tid * E;
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = j0 + i < whi ? row.at(j0 + i) : Ff{0.f, 0.f};
#pragma unroll
      for (int i = 0; i < E; ++i) {
        mine = ff_add(mine, x[i]);
        if (x[i].s > 0.f) with_mass = (int)(j0 + i);
      }
      Ff inc = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const Ff y{__shfl_up_sync(0xffffffffu, inc.s, d), __shfl_up_sync(0xffffffffu, inc.c, d)};
        if (lane >= d) inc = ff_add(inc, y);
      }
      const Ff prev{__shfl_up_sync(0xffffffffu, inc.s, 1), __shfl_up_sync(0xffffffffu, inc.c, 1)};
      if (lane == 31) sh.warp_sum[warp] = ff_value(inc);
      __syncthreads();
      if (warp == 0) {
        const double from = c0 == wlo ? sh.base : sh.warp_base[kWarps];
        const double upto = from + scan16(lane < kWarps ? sh.warp_sum[lane] : 0.0, lane);
        __syncwarp();
        if (lane == 0) sh.warp_base[0] = from;
        if (lane < kWarps) sh.warp_base[lane + 1] = upto;
      }
      __syncthreads();
      const bool ends = sh.warp_base[kWarps] > t;   // uniform
      // Should the sums of a warp's entries, added one by one, not pass t where
      // its whole sum does: its last entry, or what lies below.
      if (with_mass >= 0 && (!ends || sh.warp_base[warp] <= t)) atomicMax(&sh.last, with_mass);
      if (sh.warp_base[warp] <= t && t < sh.warp_base[warp + 1]) {
        const double mybase = sh.warp_base[warp];
        if (mybase + ff_value(inc) > t) {
          double run = mybase + (lane ? ff_value(prev) : 0.0);
#pragma unroll
          for (int i = 0; i < E; ++i) {
            run += ff_value(x[i]);
            if (x[i].s > 0.f && run > t) {
              atomicMin(&sh.found, (int)(j0 + i));
              break;
            }
          }
        }
      }
      if (ends) break;
    }
    __syncthreads();
    if (tid == 0)
      a.tokens[(long long)bb * a.w + n_acc] = sh.found != 0x7fffffff ? sh.found : sh.last;
  } else if (!(sh.total > 0.0) && rank == 0 && tid == 0) {
    a.tokens[(long long)bb * a.w + n_acc] = -1;
  }
  cl.sync();   // cta_sum stays readable until every CTA has read it
}

template <typename T>
cudaError_t run_tokens(const TokenArgs& a, int sms, cudaStream_t st) {
  // Two CTAs per SM fill the memory system; a CTA below 2048 entries would
  // only add barrier time.
  int C = 1;
  while (C < kMaxCluster && (long long)a.b * C * 2 <= 2LL * sms && a.vocab / (C * 2) >= 2048) C *= 2;
  const cudaError_t e = launch_pdl_cluster(verify_tokens_kernel<T>, dim3((unsigned)(a.b * C)),
                                           dim3(kThreads), 0, st, (unsigned)C, a);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace

cudaError_t launch_tokens(const TokenArgs& a, bool bf16, int sms, cudaStream_t st) {
  return bf16 ? run_tokens<__nv_bfloat16>(a, sms, st) : run_tokens<float>(a, sms, st);
}

cudaError_t take_tokens_flags(unsigned* flags) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_tokens_dev_flags, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_tokens_dev_flags, &zero, sizeof(zero));
  *flags |= v;
  return e;
}

}  // namespace dustin
