// Log probabilities of given tokens, entropy and the most likely alternatives of
// rows of logits.
//
// With M = max x_j, t_j = c (x_j - M), c = scale log2 e, and l = sum_j 2^t_j:
//   lse = scale M + ln l,      logprob(j) = scale (x_j - M) - ln l,
//   entropy = ln l - ln 2 / l sum_j 2^t_j t_j.
// One pass: each thread keeps (m, l, s = sum 2^t t) over its entries; two parts
// join at the larger m with
//   l = l_1 + f l_2,  s = s_1 + f (s_2 + l_2 t),  t = c (m_2 - m_1), f = 2^t.
// Differences x_j - m are formed before they are scaled, so that their rounding
// goes by their own size and not by the logits', and halved, so that those of the
// largest numbers stay finite.
//
// The alternatives are found in the same pass.  Of the first batch the `top` largest
// lane maxima give a bound that `top` entries reach; entries that reach it go to a
// list in shared memory, which after the first batch is cut to its `top` best, the
// last of which is the next bound: some top * ln(row / batch) entries follow, taken
// without a barrier.  (That and entries taken in pairs: 249 -> 191 us for a prompt's
// rows; batches kept as they are read and the bound raised only where the list grew:
// 176.)  Should they not fit (rows that rise, or have few values above many equal
// ones), the list's own `top`-th is a bound for a second pass, which cuts the list as it
// fills.  An entry that equals a bound counts if its index is lower, so ties go to the
// lowest index and equal entries (banned tokens at -inf) do not fill the list.  But each
// of them is read again and compared by its index, one at a time: where the bound is
// -inf or a value that most of the row has, that is most of the time (a prompt's rows with
// all but 10 tokens banned: 565 us with one alternative, 1107 with 20; with all but
// 1000 banned as without).  Places come from counting better entries: no order of
// atomics shows.
//
// One cluster of C CTAs per row (C by the number of rows); rank 0 joins the parts
// through distributed shared memory.  No workspace.  Many rows: no
// pipe is full (issue 65 %, arithmetic 42 %, DRAM 45 %; 14.6 instructions a logit, of
// which the sums need some 6; stalls: barriers, waits of a few cycles).  Few: the
// latency of a load batch, three barriers, the cluster's.
//
// Measured (2048 rows of 152064 in bf16, 623 MB): 173 us with one alternative, 3.6
// TB/s; 136 without any, 4.6 TB/s; 217 with 20; in fp32 212 and 198, 5.9 and 6.3 TB/s.
// 4 rows of 32000 in fp32: 9.2 us.
#include <algorithm>
#include <climits>
#include <cooperative_groups.h>

#include "device_common.cuh"
#include "dustin.h"
#include "internal.h"

namespace cg = cooperative_groups;

namespace dustin {

namespace {

__device__ unsigned int g_logprobs_dev_flags;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kWords = 4;                   // 16-byte words of a thread per batch
constexpr int kTop = kLogprobsMaxTop;
constexpr int kLists = (kTop + kWarps - 1) / kWarps;   // lane maxima a warp gives
constexpr int kList = 1024;
constexpr int kRefine = 192;                // entries that a list may keep between batches
static_assert(kRefine + kThreads <= kList && kMaxCluster * kTop <= kList, "list");

// Two fp32 numbers at a time.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float lo_of(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float hi_of(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

using Key = unsigned long long;             // larger: better

// Order of values as unsigned numbers; -0 counts as +0.
__device__ __forceinline__ unsigned order_of(float x) {
  const unsigned u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ Key key_of(float x, int j) {
  return (Key)order_of(x) << 32 | (unsigned)~j;
}
__device__ __forceinline__ int index_of(Key k) { return (int)~(unsigned)k; }

struct Sums {
  float m, l, s;
};
// c (x - m) from half, -m / 2, and c2, 2 c.
__device__ __forceinline__ float exponent(float x, float half, float c2) {
  return fmaf(x, 0.5f, half) * c2;
}
// 2^t times t where 2^t is 0: 0, though t be -inf.
constexpr float kLeast = -1e30f;

// l of a part without entries above -inf is 0, or NaN where it met one.
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b, float c2) {
  Sums r;
  r.m = fmaxf(a.m, b.m);
  r.l = a.l + b.l;
  r.s = 0.f;
  if (r.m == -INFINITY) return r;
  r.l = 0.f;
  const Sums* part[2] = {&a, &b};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const Sums& p = *part[i];
    if (p.m == -INFINITY) {
      r.l += p.l;
    } else {
      const float t = fmaxf(exponent(p.m, -0.5f * r.m, c2), kLeast), f = ex2(t);
      r.l = fmaf(f, p.l, r.l);
      r.s = fmaf(f, fmaf(p.l, t, p.s), r.s);
    }
  }
  return r;
}

// sum += x, with what the roundings so far have added too much in `over` (Kahan): a
// thread of a long row adds thousands of batches, each of which may be less than half a
// step of the sum.  (One sum over all entries lost 2e-4 of 2^26 of them, 3e-3 of 2^30.)
__device__ __forceinline__ void add_up(float& sum, float& over, float x) {
  const float y = __fsub_rn(x, over), t = __fadd_rn(sum, y);
  over = __fsub_rn(__fsub_rn(t, sum), y);
  sum = t;
}

struct Shared {
  alignas(16) Key list[kList];
  Key best[kTop];
  unsigned maxima[kWarps * kLists];
  Sums part[kWarps], all;
  Key bound;
  int count, over, kept;
};

// The list's `top` best to sh.best in order, and back to the list's start.  All
// threads; the list is complete and stays so.
__device__ void refine(Shared& sh, int top) {
  __syncthreads();
  const int n = min(sh.count, kList);
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const Key mine = sh.list[i];
    int better = 0;
    for (int j = 0; j < n; ++j) better += sh.list[j] > mine;
    if (better < top) sh.best[better] = mine;
  }
  __syncthreads();
  const int kept = min(n, top);
  if (threadIdx.x < kept) sh.list[threadIdx.x] = sh.best[threadIdx.x];
  if (threadIdx.x == 0) {
    sh.count = sh.kept = kept;
    if (kept == top) sh.bound = sh.best[top - 1];
  }
  __syncthreads();
}

template <typename T>
__device__ __forceinline__ float element(const uint4& w, int i) {
  const uint32_t* u = &w.x;
  if constexpr (sizeof(T) == 4) return __uint_as_float(u[i]);
  return __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
}

// Makes an entry -inf.
template <typename T>
__device__ __forceinline__ void forget(uint4& w, int i) {
  uint32_t* u = &w.x;
  if constexpr (sizeof(T) == 4)
    u[i] = 0xff800000u;
  else
    u[i / 2] = i & 1 ? (u[i / 2] & 0xffffu) | 0xff800000u : (u[i / 2] & 0xffff0000u) | 0xff80u;
}
// The largest entry that is not NaN, or -inf.
template <typename T>
__device__ __forceinline__ float largest(const uint4 (&w)[kWords]) {
  if constexpr (sizeof(T) == 4) {
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < kWords; ++u) {
      m = max3(m, __uint_as_float(w[u].x), __uint_as_float(w[u].y));
      m = max3(m, __uint_as_float(w[u].z), __uint_as_float(w[u].w));
    }
    return m;
  } else {
    uint32_t m = 0xff80ff80u;                            // two -inf
#pragma unroll
    for (int u = 0; u < kWords; ++u) {
      const uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) asm("max.bf16x2 %0, %0, %1;\n" : "+r"(m) : "r"(x[i]));
    }
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
    logprobs_kernel(const __grid_constant__ LogprobArgs a) {
  constexpr int V = 16 / sizeof(T);                    // entries of 16 bytes
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
  const int row = blockIdx.x / ranks, bb = row / a.w, t = row - bb * a.w;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float c2 = 2.f * a.scale * kLog2e;
  const int top = a.top;
  griddep_wait();
  griddep_launch_dependents();
  if (a.n_rows && t >= __ldg(a.n_rows + bb)) return;   // the whole cluster
  const T* x = static_cast<const T*>(a.x) + bb * a.stride_b + t * a.stride_w;
  // The logit of a given token, fetched ahead.
  int token = 0;
  float given = -INFINITY;
  if (rank == 0 && tid < a.m) {
    token = __ldg(a.tokens + (long long)row * a.m + tid);
    if (token >= 0 && token < a.vocab)
      given = (float)x[token];
    else if (token != -1)
      atomicOr(&g_logprobs_dev_flags, DUSTIN_DEVFLAG_INDEX_RANGE);
  }
  if (tid == 0) {
    sh.count = sh.over = sh.kept = 0;
    sh.bound = 0;                                      // every entry but NaN is better
  }
  // Words of 16 bytes; entry i of word k is entry k V + i - lead of the row.
  const int lead = (int)(reinterpret_cast<uintptr_t>(x) & 15u) / (int)sizeof(T);
  const uint4* words = reinterpret_cast<const uint4*>(x - lead);
  const long long all = ((long long)lead + a.vocab + V - 1) / V;
  const int w0 = (int)(all * rank / ranks), w1 = (int)(all * (rank + 1) / ranks);
  const int last = (int)all - 1;

  Sums sum{-INFINITY, 0.f, 0.f};
  float l_over = 0.f, s_over = 0.f;                    // what their roundings added
  uint4 next[kWords];
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < kWords; ++u) {
      const int k = base + u * kThreads + tid;
      if (k < w1) next[u] = __ldg(words + k);
    }
  };
  constexpr int kStep = kThreads * kWords;
  for (int pass = 0; pass < 2; ++pass) {
    load(w0);
    __syncthreads();
    for (int base = w0, batch = 0; base < w1; base += kStep, ++batch) {
      uint4 cur[kWords];
      auto v = [&](int u, int i) { return element<T>(cur[u], i); };
#pragma unroll
      for (int u = 0; u < kWords; ++u) {
        const int k = base + u * kThreads + tid;
        cur[u] = next[u];
        if (k == 0 || k >= last || k >= w1) {            // entries beside the row, or none
          const long long j0 = (long long)k * V - lead;
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (k >= w1 || j0 + i < 0 || j0 + i >= a.vocab) forget<T>(cur[u], i);
        }
      }
      load(base + kStep);
      const float most = largest<T>(cur);
      if (pass == 0) {
        if (most > sum.m) {
          const float t = fmaxf(exponent(sum.m, -0.5f * most, c2), kLeast), f = ex2(t);
          sum.s = f * fmaf(sum.l, t, sum.s);
          sum.l *= f;
          sum.m = most;
          l_over *= f;
          s_over *= f;
        }
        const float half = sum.m == -INFINITY ? 0.f : -0.5f * sum.m;
        const uint64_t half2 = pack2(half, half), scale2 = pack2(c2, c2), point5 = pack2(0.5f, 0.5f);
        uint64_t l2 = 0, s2 = 0;
#pragma unroll
        for (int u = 0; u < kWords; ++u)
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            // exponent(), two entries at a time
            const uint64_t t = mul2(fma2(pack2(v(u, i), v(u, i + 1)), point5, half2), scale2);
            const uint64_t e = pack2(ex2(lo_of(t)), ex2(hi_of(t)));
            l2 = add2(l2, e);
            s2 = fma2(e, pack2(fmaxf(lo_of(t), kLeast), fmaxf(hi_of(t), kLeast)), s2);
          }
        add_up(sum.l, l_over, lo_of(l2) + hi_of(l2));
        add_up(sum.s, s_over, lo_of(s2) + hi_of(s2));
      }
      if (top == 0) continue;

      if (base == w0 && pass == 0) {
        // A first bound: the `top`-th of the warps' best lane maxima.
        unsigned mine = order_of(most);
        const int lists = (top + kWarps - 1) / kWarps;
        for (int i = 0; i < lists; ++i) {
          const unsigned best = __reduce_max_sync(0xffffffffu, mine);
          if (lane == 0) sh.maxima[warp * lists + i] = best;
          const unsigned has = __ballot_sync(0xffffffffu, mine == best);
          if (lane == __ffs(has) - 1) mine = 0;
        }
        __syncthreads();
        const int n = kWarps * lists;
        if (tid < n) {
          const unsigned x0 = sh.maxima[tid];
          int better = 0;
          for (int i = 0; i < n; ++i) better += sh.maxima[i] > x0 || (sh.maxima[i] == x0 && i < tid);
          // Entries equal to it count, whatever their index; -inf bounds nothing
          // (lanes without an entry have it, too).
          if (better == top - 1 && value_of(x0) > -INFINITY) sh.bound = (Key)x0 << 32;
        }
        __syncthreads();
        // Rows with few words leave warps with too few: of all lanes, then.
        if (sh.bound == 0) {
          unsigned* lanes = reinterpret_cast<unsigned*>(sh.list);   // still empty
          const unsigned x0 = order_of(most);
          lanes[tid] = x0;
          __syncthreads();
          int better = 0;
          for (int i = 0; i < kThreads; i += 4) {
            const uint4 y = *reinterpret_cast<const uint4*>(lanes + i);
            better += y.x > x0 || (y.x == x0 && i < tid);
            better += y.y > x0 || (y.y == x0 && i + 1 < tid);
            better += y.z > x0 || (y.z == x0 && i + 2 < tid);
            better += y.w > x0 || (y.w == x0 && i + 3 < tid);
          }
          __syncthreads();                               // the list may be filled
          if (better == top - 1 && value_of(x0) > -INFINITY) sh.bound = (Key)x0 << 32;
          __syncthreads();
        }
      }
      // Entries that reach the bound.  It rises after 1, 2, 4, .. batches.
      const bool apart = base > w0 && pass == 0;           // no barriers
      if (apart && !(batch & (batch - 1)) && __syncthreads_or(sh.count > top)) refine(sh, top);
      Key bound = sh.bound;
      float least = bound ? value_of((unsigned)(bound >> 32)) : -INFINITY;
      // Entry e of the thread's, read again from the row; 0: none that counts.
      auto entry = [&](int e) -> Key {
        const int k = base + e / V * kThreads + tid;
        const long long j = (long long)k * V + e % V - lead;
        if (k >= w1 || j < 0 || j >= a.vocab) return 0;
        const float xv = (float)x[j];
        if (!(xv >= least)) return 0;
        const Key key = key_of(xv, (int)j);
        return key > bound ? key : 0;
      };
      int before = 0;
      if (!apart) {
        before = sh.count;
        __syncthreads();                                   // all have read the count
      }
      if (most >= least) {
        unsigned reach = 0;
#pragma unroll
        for (int u = 0; u < kWords; ++u)
#pragma unroll
          for (int i = 0; i < V; ++i) reach |= (unsigned)(v(u, i) >= least) << (u * V + i);
        while (reach) {          // few, unless the bound is a value of most entries
          const Key key = entry(__ffs(reach) - 1);
          reach &= reach - 1;
          if (!key) continue;
          const int at = atomicAdd(&sh.count, 1);
          if (at < kList)
            sh.list[at] = key;
          else
            sh.over = 1;
        }
      }
      if (apart) continue;
      __syncthreads();
      if (sh.over) {
        // Taken again, one word and entry at a time, the list cut in between.
        __syncthreads();
        if (tid == 0) sh.count = before, sh.over = 0;      // at most kRefine
        __syncthreads();
#pragma unroll 1
        for (int e = 0; e < kWords * V; ++e) {
          const Key key = entry(e);
          if (__syncthreads_or(key != 0)) {
            if (key) sh.list[atomicAdd(&sh.count, 1)] = key;
            refine(sh, top);
            bound = sh.bound;
            least = bound ? value_of((unsigned)(bound >> 32)) : -INFINITY;
          }
        }
      } else if (sh.count > kRefine || base == w0) {
        refine(sh, top);
      }
    }
    __syncthreads();
    const bool again = sh.over;                          // in the first pass only
    if (top > 0) refine(sh, top);
    if (!again) break;
    // A second pass: the bound is kept, the list is not.
    if (tid == 0) {
      sh.bound = sh.best[top - 1] - 1;                     // reached by that one, too
      sh.count = sh.over = 0;
    }
    __syncthreads();
  }

  // Sums: lanes, warps, CTAs.
  sum.l -= l_over;
  sum.s -= s_over;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const Sums o{__shfl_xor_sync(0xffffffffu, sum.m, d), __shfl_xor_sync(0xffffffffu, sum.l, d),
                 __shfl_xor_sync(0xffffffffu, sum.s, d)};
    sum = lane & d ? join(o, sum, c2) : join(sum, o, c2);
  }
  if (lane == 0) sh.part[warp] = sum;
  __syncthreads();
  if (tid == 0) {
    Sums r = sh.part[0];
    for (int i = 1; i < kWarps; ++i) r = join(r, sh.part[i], c2);
    sh.all = r;
  }
  if (ranks > 1) {
    cluster.sync();
    if (rank == 0) {
      if (tid == 0) {
        Sums r = sh.all;
        for (int i = 1; i < ranks; ++i) r = join(r, *cluster.map_shared_rank(&sh.all, i), c2);
        sh.all = r;
      }
      for (int i = tid; i < (ranks - 1) * top; i += kThreads) {
        const Shared* of = cluster.map_shared_rank(&sh, 1 + i / top);
        if (i % top < of->kept) sh.list[atomicAdd(&sh.count, 1)] = of->best[i % top];
      }
    }
    cluster.sync();                                    // the others' parts are read
    if (rank) return;
    if (top > 0) refine(sh, top);
  }
  __syncthreads();
  const Sums r = sh.all;
  const bool none = r.m == -INFINITY && r.l == 0.f;    // only -inf
  const float ln_l = none ? 0.f : logf(r.l);           // NaN where an entry is NaN or +inf
  auto logprob = [&](float xv) {
    return none ? -INFINITY : isnan(ln_l) ? ln_l : fmaf(xv, 0.5f, -0.5f * r.m) * (2.f * a.scale) - ln_l;
  };
  if (tid < a.m) a.logprobs[(long long)row * a.m + tid] = logprob(given);
  if (tid < top) {
    const bool have = tid < sh.kept;                   // NaN entries are no alternatives
    const Key key = have ? sh.best[tid] : 0;
    a.top_ids[(long long)row * top + tid] = have ? index_of(key) : -1;
    a.top_logprobs[(long long)row * top + tid] =
        have ? logprob(value_of((unsigned)(key >> 32))) : NAN;
  }
  if (tid == 0) {
    if (a.entropy) a.entropy[row] = none ? 0.f : ln_l - kLn2 * r.s / r.l;
    if (a.lse) a.lse[row] = none ? -INFINITY : isnan(ln_l) ? ln_l : fmaf(r.m, a.scale, ln_l);
  }
}

template <typename T>
cudaError_t run(const LogprobArgs& a, int sms, cudaStream_t st) {
  // CTAs per row: twice the SMs in all, and a load batch of each CTA's at least
  // one word per thread.
  const long long rows = (long long)a.b * a.w;
  const long long words = (a.vocab + 16 / sizeof(T) - 1) / (16 / sizeof(T));
  int c = 1;
  while (c < kMaxCluster && rows * c < 2 * sms && words > (long long)c * kThreads) c *= 2;
  const dim3 grid((unsigned)(rows * c)), block(kThreads);
  cudaError_t e = c == 1 ? launch_pdl(logprobs_kernel<T>, grid, block, 0, st, a)
                         : launch_pdl_cluster(logprobs_kernel<T>, grid, block, 0, st, c, a);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, bool bf16, int sms, cudaStream_t st) {
  return bf16 ? run<__nv_bfloat16>(a, sms, st) : run<float>(a, sms, st);
}

cudaError_t take_logprobs_flags(unsigned* flags) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_logprobs_dev_flags, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_logprobs_dev_flags, &zero, sizeof(zero));
  *flags |= v;
  return e;
}

}  // namespace dustin
