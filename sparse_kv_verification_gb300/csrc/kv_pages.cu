// Cache bookkeeping around a verification step: compaction of a cache to an
// index set, and pages shared between sequences (fork, grow with copy on
// write, release).
//
//  * kv_compact_kernel: one CTA per (layer, sequence, kv head) and range of
//    kept positions, 128 rows of K and V at a time: the offsets of the next
//    rows (index, then page table) are fetched while the current rows move,
//    and a thread holds its 16-byte pieces of all rows of the chunk in
//    registers between loads and stores.  Bound by HBM (each kept row is
//    read and written once).  In place, one CTA walks the whole kept list:
//    with ascending indices, row i comes from a position >= i, so a chunk's
//    stores never touch a row that a later chunk still has to read, and
//    within a chunk a barrier stands between the last load and the first
//    store.  Measured: 2048 of 32768 positions of 16 sequences, four layers of
//    8 heads, 167 us (1.07 GB moved, 6.4 TB/s); 512 of 8192 in place on pages
//    of 16, four layers of 4 sequences and heads, 10.4 us (64 CTAs, the
//    latency of four chunks).
//  * kv_fork_kernel: one CTA per fork; table row copied, counts raised.
//  * kv_resize_kernel: one cluster of 8 CTAs (for small pools and lists one CTA
//    of 256 threads) does the whole update of the table, the lengths and the
//    reference counts (a few microseconds of latency, far from any bandwidth):
//    each CTA derives the same plan from the list, releases its share of the
//    dropped entries, and reads its slice of the reference counts into a bitmap
//    of free pages; ranks in page order come from population counts, so the
//    pages given out do not depend on timing.
//  * kv_copy_pages_kernel: the copies that growth into a shared page asks
//    for, one CTA per (list entry, layer, K or V).
// Measured, a turn of a serving loop (release, fork, grow with its copies): 64
// samples of four prompts of 32749 positions on pages of 16, four layers of 8
// heads, 36.2 us; four samples of one prompt of 2051 13.5.  Every launch is
// bound by its latency: the pages' rows copied take 0.6 us of bandwidth.
#include <algorithm>
#include <cooperative_groups.h>

#include "device_common.cuh"
#include "dustin.h"
#include "internal.h"

namespace cg = cooperative_groups;

namespace dustin {

namespace {

__device__ unsigned int g_pages_dev_flags;

__device__ __forceinline__ void raise_flag(unsigned f) { atomicOr(&g_pages_dev_flags, f); }

// ---- compaction

constexpr int kCompactThreads = 256;
constexpr int kChunk = 128;   // rows moved at a time

// Element offset of position j of sequence bb, kv head h; -1 if its page id
// lies outside the pool.
__device__ __forceinline__ long long row_offset(const KvView& kv, int bb, int h, int j) {
  if (!kv.page_table)
    return (long long)bb * kv.sb + (long long)h * kv.sh + (long long)j * kv.sn;
  const int pg = __ldg(kv.page_table + (long long)bb * kv.pages_per_seq + j / kv.page_size);
  if (pg < 0 || pg >= kv.num_pages) return -1;
  return (long long)pg * kv.sb + (long long)h * kv.sh + (long long)(j % kv.page_size) * kv.sn;
}

template <int D>
__global__ void __launch_bounds__(kCompactThreads)
    kv_compact_kernel(const __grid_constant__ CompactArgs a) {
  constexpr int LPR = D / 8;                          // lanes per row
  constexpr int RPP = kCompactThreads / LPR;          // rows per pass
  constexpr int U = kChunk / RPP;                     // passes per chunk
  __shared__ long long soff[2][kChunk], doff[2][kChunk];
  const int tid = threadIdx.x;
  const int split = blockIdx.x % a.splits;
  const int unit = blockIdx.x / a.splits;
  const int h = unit % a.hkv, bb = unit / a.hkv % a.b, layer = unit / a.hkv / a.b;
  const KvView& src = a.layer[layer].src;
  const KvView& dst = a.layer[layer].dst;
  griddep_wait();
  griddep_launch_dependents();
  int kept = a.k;
  if (a.k_len) kept = min(max(__ldg(a.k_len + bb), 0), a.k);
  const int per = (a.k + a.splits * kChunk - 1) / (a.splits * kChunk) * kChunk;
  const int i0 = min(split * per, kept), i1 = min(i0 + per, kept);
  const int* idx = a.idx + (long long)bb * a.k;

  auto offsets = [&](int buf, int first) {
    if (tid >= kChunk) return;
    long long so = -1, to = -1;
    const int i = first + tid;
    if (i < i1) {
      const int j = __ldg(idx + i);
      if (j < 0 || j >= a.n) {
        raise_flag(DUSTIN_DEVFLAG_INDEX_RANGE);
      } else {
        if (a.in_place && i > 0 && __ldg(idx + i - 1) >= j) raise_flag(DUSTIN_DEVFLAG_INDEX_ORDER);
        so = row_offset(src, bb, h, j);
        to = row_offset(dst, bb, h, i);
        if (so < 0 || to < 0) raise_flag(DUSTIN_DEVFLAG_PAGE_RANGE);
        if (a.in_place && so == to) so = -1;   // already where it belongs
      }
    }
    soff[buf][tid] = to < 0 ? -1 : so;
    doff[buf][tid] = to;
  };

  const int lr = tid / LPR, lc = tid % LPR * 8;
  offsets(0, i0);
  __syncthreads();
  int buf = 0;
  for (int c = i0; c < i1; c += kChunk, buf ^= 1) {
    uint4 kr[U], vr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long so = soff[buf][u * RPP + lr];
      if (so >= 0) {
        kr[u] = *reinterpret_cast<const uint4*>(src.k + so + lc);
        vr[u] = *reinterpret_cast<const uint4*>(src.v + so + lc);
      }
    }
    if (c + kChunk < i1) offsets(buf ^ 1, c + kChunk);
    // In place, every load of the chunk is in registers before a store.
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (soff[buf][u * RPP + lr] >= 0) {
        const long long to = doff[buf][u * RPP + lr];
        *reinterpret_cast<uint4*>(const_cast<__nv_bfloat16*>(dst.k) + to + lc) = kr[u];
        *reinterpret_cast<uint4*>(const_cast<__nv_bfloat16*>(dst.v) + to + lc) = vr[u];
      }
    }
    __syncthreads();   // this buffer's offsets are rewritten two chunks on
  }
}

// ---- fork

constexpr int kForkThreads = 256;

__global__ void __launch_bounds__(kForkThreads) kv_fork_kernel(const ForkArgs a) {
  __shared__ int bad;
  const int f = blockIdx.x, tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const int p = __ldg(a.parent + f), c = __ldg(a.child + f);
  const int cap = a.pages_per_seq * a.page_size;
  const bool in_range = p >= 0 && p < a.n_seqs && c >= 0 && c < a.n_seqs && p != c;
  int plen = 0;
  if (tid == 0) {
    bad = !in_range;
    if (in_range) {
      plen = a.seq_len[p];
      if (a.seq_len[c] != 0 || plen < 0 || plen > cap) bad = 1;
    }
  }
  __syncthreads();
  // A child named before, or a parent that is itself a child of this call.
  for (int j = tid; j < a.n_forks; j += kForkThreads) {
    const int cj = __ldg(a.child + j);
    if ((j < f && cj == c) || cj == p) bad = 1;
  }
  __syncthreads();
  if (bad) {
    if (tid == 0) raise_flag(DUSTIN_DEVFLAG_INDEX_RANGE);
    return;
  }
  plen = a.seq_len[p];
  const int pages = (plen + a.page_size - 1) / a.page_size;
  const int* from = a.page_table + (long long)p * a.pages_per_seq;
  int* to = a.page_table + (long long)c * a.pages_per_seq;
  for (int i = tid; i < pages; i += kForkThreads) {
    const int pg = from[i];
    to[i] = pg;
    if (pg >= 0 && pg < a.num_pages)
      atomicAdd(a.refcount + pg, 1);
    else
      raise_flag(DUSTIN_DEVFLAG_PAGE_RANGE);
  }
  if (tid == 0) a.seq_len[c] = plen;
}

// ---- resize

constexpr int kResizeThreads = 1024;
constexpr int kResizeCluster = 8;
constexpr int kDropBlock = 256;   // table entries a warp drops at a time

constexpr int kNames = 2 * kResizeMaxList;   // a power of two, half empty

struct ResizeShared {
  int seq[kResizeMaxList];
  int name[kNames], first_named[kNames];   // sequences by hash, their first entries
  int had[kResizeMaxList];      // pages before; -1: entry left out
  int have[kResizeMaxList];     // pages after
  int last[kResizeMaxList];     // last page to be copied (-1: none)
  int first[kResizeMaxList];    // rank of the entry's first free page
  int scan[32];
  int free_here;                // read by the other CTAs of the cluster
  int total;
  int base, free_all;
};

// Exclusive sum of v over the CTA's threads; *total receives the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += y;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  const int mine = lane < warps ? warp_sums[lane] : 0;
  int w = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += y;
  }
  const int below = __shfl_sync(0xffffffffu, w - mine, warp);
  const int all = __shfl_sync(0xffffffffu, w, 31);
  if (threadIdx.x == 0) *total = all;
  __syncthreads();   // also: warp_sums may be written again
  return below + inc - v;
}

__global__ void __launch_bounds__(kResizeThreads) kv_resize_kernel(const ResizeArgs a) {
  extern __shared__ unsigned bitmap[];   // free pages of this CTA's slice
  __shared__ ResizeShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), C = (int)cl.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = blockDim.x, warps = threads >> 5;
  griddep_wait();
  griddep_launch_dependents();

  // The plan, the same in every CTA.
  const long long cap = (long long)a.pages_per_seq * a.page_size;
  int old = 0, now = 0, seq = -1;
  bool ok = false;
  for (int i = tid; i < kNames; i += threads) {
    sh.name[i] = -1;
    sh.first_named[i] = kResizeMaxList;
  }
  __syncthreads();
  int at = 0;
  if (tid < a.n_list) {
    seq = __ldg(a.seqs + tid);
    sh.seq[tid] = seq;
    ok = seq >= 0 && seq < a.n_seqs;
    if (ok) {
      // Its place: the next free one from its hash (1024 names leave half of
      // them free).  Comparing with every entry before took 10 us of 1024.
      at = (int)(((unsigned)seq * 2654435761u) >> 16) & (kNames - 1);
      for (int i = 0; i < kNames; ++i, at = (at + 1) & (kNames - 1)) {
        const int there = atomicCAS(&sh.name[at], -1, seq);
        if (there == -1 || there == seq) break;
      }
      atomicMin(&sh.first_named[at], tid);
      now = a.new_len ? __ldg(a.new_len + tid) : 0;
      old = __ldcg(a.seq_len + seq);
      ok = now >= 0 && now <= cap && old >= 0 && old <= cap;
    }
  }
  __syncthreads();
  if (tid < a.n_list) {
    if (ok && sh.first_named[at] != tid) ok = false;
    if (!ok && rank == 0) raise_flag(DUSTIN_DEVFLAG_INDEX_RANGE);
    sh.had[tid] = ok ? (old + a.page_size - 1) / a.page_size : -1;
    sh.have[tid] = (now + a.page_size - 1) / a.page_size;
  }
  __syncthreads();

  // Entries behind the new ends, in blocks dealt to all warps of the cluster.
  const int per_entry = (a.pages_per_seq + kDropBlock - 1) / kDropBlock;
  for (int x = rank * warps + warp; x < a.n_list * per_entry; x += C * warps) {
    const int i = x / per_entry, s0 = (x - i * per_entry) * kDropBlock;
    const int lo = max(sh.have[i], s0), hi = min(sh.had[i], s0 + kDropBlock);
    if (lo >= hi) continue;
    int* row = a.page_table + (long long)sh.seq[i] * a.pages_per_seq;
    int pg[kDropBlock / 32];
#pragma unroll
    for (int u = 0; u < kDropBlock / 32; ++u) {
      const int s = lo + u * 32 + lane;
      pg[u] = s < hi ? row[s] : -1;
    }
#pragma unroll
    for (int u = 0; u < kDropBlock / 32; ++u) {
      const int s = lo + u * 32 + lane;
      if (s >= hi) continue;
      if (pg[u] >= 0 && pg[u] < a.num_pages)
        atomicSub(a.refcount + pg[u], 1);
      else
        raise_flag(DUSTIN_DEVFLAG_PAGE_RANGE);
      row[s] = -1;
    }
  }
  cl.sync();

  // Pages wanted, in list order: the copy of a shared partial page first.
  int need = 0, last = -1;
  if (tid < a.n_list && ok && now > old) {
    const int had = sh.had[tid];
    need = sh.have[tid] - had;
    if (old % a.page_size) {
      const int pg = __ldcg(a.page_table + (long long)seq * a.pages_per_seq + had - 1);
      if (pg < 0 || pg >= a.num_pages) {
        if (rank == 0) raise_flag(DUSTIN_DEVFLAG_PAGE_RANGE);
      } else if (__ldcg(a.refcount + pg) > 1) {
        last = pg;
        ++need;
      }
    }
  }
  const int first = block_scan(need, sh.scan, &sh.total);
  if (tid < a.n_list) {
    sh.first[tid] = first;
    sh.last[tid] = last;
  }
  const int wanted = sh.total;
  int free_all = 0;
  if (wanted > 0) {   // uniform over the cluster
    const int per = ((a.num_pages + C - 1) / C + 31) / 32 * 32;
    const int lo = min(rank * per, a.num_pages), hi = min(lo + per, a.num_pages);
    const int words = (hi - lo + 31) / 32;
#pragma unroll 8
    for (int wd = warp; wd < words; wd += warps) {
      const int pg = lo + wd * 32 + lane;
      const bool is_free = pg < hi && __ldcg(a.refcount + pg) == 0;
      const unsigned bits = __ballot_sync(0xffffffffu, is_free);
      if (lane == 0) bitmap[wd] = bits;
    }
    __syncthreads();
    const int m = (words + threads - 1) / threads;
    const int w0 = min(tid * m, words), w1 = min(w0 + m, words);
    int count = 0;
    for (int wd = w0; wd < w1; ++wd) count += __popc(bitmap[wd]);
    int r = block_scan(count, sh.scan, &sh.free_here);
    cl.sync();
    if (warp == 0) {
      const int c = lane < C ? *cl.map_shared_rank(&sh.free_here, lane) : 0;
      int inc = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
      }
      if (lane == rank) sh.base = inc - c;
      if (lane == 31) sh.free_all = inc;
    }
    __syncthreads();
    free_all = sh.free_all;
    r += sh.base;
    // A warp gives out its threads' words one after another, a lane to a page:
    // the free pages of the lowest numbers often lie in a few words.
    unsigned todo = __ballot_sync(0xffffffffu, count > 0 && r < wanted);
    while (todo) {
      const int src = __ffs((int)todo) - 1;
      todo &= todo - 1;
      int before = __shfl_sync(0xffffffffu, r, src);
      const int s0 = __shfl_sync(0xffffffffu, w0, src), s1 = __shfl_sync(0xffffffffu, w1, src);
      for (int wd = s0; wd < s1 && before < wanted; ++wd) {
        const unsigned bits = bitmap[wd];
        const int mine = before + __popc(bits & ((1u << lane) - 1));
        before += __popc(bits);
        if (!(bits >> lane & 1) || mine >= wanted) continue;
        const int pg = lo + wd * 32 + lane;
        // The entry whose ranks hold it: the last with first <= mine.  Entries
        // without need share their first with the next one, which is later.
        int x = 0, y = a.n_list - 1;
        while (x < y) {
          const int mid = (x + y + 1) >> 1;
          if (sh.first[mid] <= mine)
            x = mid;
          else
            y = mid - 1;
        }
        const int end = x + 1 < a.n_list ? sh.first[x + 1] : wanted;
        if (end <= free_all) {   // the whole entry is served
          const int cow = sh.last[x] >= 0 ? 1 : 0;
          const int slot = mine - sh.first[x] - cow;
          a.page_table[(long long)sh.seq[x] * a.pages_per_seq + sh.had[x] + slot] = pg;
          a.refcount[pg] = 1;
          if (slot < 0) {
            a.copies[2 * x] = sh.last[x];
            a.copies[2 * x + 1] = pg;
          }
        }
      }
    }
  }
  if (rank == 0 && tid < a.n_list) {
    const bool served = ok && first + need <= free_all;
    if (ok && need > 0 && !served) raise_flag(DUSTIN_DEVFLAG_NO_PAGES);
    if (ok && (need == 0 || served)) {
      a.seq_len[seq] = now;
      if (last >= 0) atomicSub(a.refcount + last, 1);
    }
    if (last < 0 || !served) a.copies[2 * tid] = a.copies[2 * tid + 1] = -1;
  }
  cl.sync();   // free_here stays readable until every CTA has read it
}

constexpr int kCopyThreads = 256;

template <int D>
__global__ void __launch_bounds__(kCopyThreads)
    kv_copy_pages_kernel(const __grid_constant__ CopyArgs a) {
  constexpr int LPR = D / 8, RPP = kCopyThreads / LPR, U = 8;
  griddep_wait();
  griddep_launch_dependents();
  const int from = __ldg(a.copies + 2 * blockIdx.x), to = __ldg(a.copies + 2 * blockIdx.x + 1);
  if (from < 0 || to < 0) return;
  const KvView& kv = a.kv[blockIdx.y >> 1];
  __nv_bfloat16* base = const_cast<__nv_bfloat16*>(blockIdx.y & 1 ? kv.v : kv.k);
  const int rows = a.hkv * kv.page_size;
  const int lr = threadIdx.x / LPR, lc = threadIdx.x % LPR * 8;
  for (int r0 = lr; r0 < rows; r0 += RPP * U) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPP;
      if (r < rows)
        x[u] = *reinterpret_cast<const uint4*>(base + (long long)from * kv.sb +
                                               (long long)(r / kv.page_size) * kv.sh +
                                               (long long)(r % kv.page_size) * kv.sn + lc);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPP;
      if (r < rows)
        *reinterpret_cast<uint4*>(base + (long long)to * kv.sb +
                                  (long long)(r / kv.page_size) * kv.sh +
                                  (long long)(r % kv.page_size) * kv.sn + lc) = x[u];
    }
  }
}

}  // namespace

cudaError_t launch_compact(const CompactArgs& args, int d, int sms, cudaStream_t st) {
  CompactArgs a = args;
  const long long units = (long long)a.layers * a.b * a.hkv;
  const int chunks = std::max(1, (a.k + kChunk - 1) / kChunk);
  // Out of place a unit is cut so that about three CTAs (192 KB of loads in
  // flight) share an SM; in place its chunks have an order.
  a.splits = a.in_place ? 1 : (int)std::min<long long>(chunks, std::max<long long>(1, (3LL * sms + units - 1) / units));
  const dim3 grid((unsigned)(units * a.splits));
  const cudaError_t e = d == 64 ? launch_pdl(kv_compact_kernel<64>, grid, dim3(kCompactThreads), 0, st, a)
                                : launch_pdl(kv_compact_kernel<128>, grid, dim3(kCompactThreads), 0, st, a);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

cudaError_t launch_fork(const ForkArgs& a, cudaStream_t st) {
  const cudaError_t e = launch_pdl(kv_fork_kernel, dim3((unsigned)a.n_forks), dim3(kForkThreads), 0, st, a);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

cudaError_t launch_resize(const ResizeArgs& a, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ensure_smem_attr(kv_resize_kernel, kResizeMaxPages / kResizeCluster / 8, done);
  if (e != cudaSuccess) return e;
  // A small update runs in one CTA, whose barriers cost less than a cluster's.
  // Measured, 8 entries grown by a page and released: of 1024 pages 8.4 us in
  // one CTA, 9.3 in the cluster, of 4096 10.9 and 9.3; 32 entries of 1024 pages
  // 10.5 and 9.7.  Nothing between was measured: the border is the last point
  // at which one CTA is known to win.
  const bool small = a.num_pages <= 1024 && a.n_list <= 16 && (long long)a.n_list * a.pages_per_seq <= 8192;
  const int C = small ? 1 : kResizeCluster;
  const int threads = small ? 256 : kResizeThreads;
  const int words = ((a.num_pages + C - 1) / C + 31) / 32;
  e = launch_pdl_cluster(kv_resize_kernel, dim3((unsigned)C), dim3((unsigned)threads),
                         (size_t)words * sizeof(unsigned), st, (unsigned)C, a);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

cudaError_t launch_copy_pages(const CopyArgs& a, int n_list, int d, cudaStream_t st) {
  const dim3 grid((unsigned)n_list, (unsigned)(2 * a.layers));
  const cudaError_t e = d == 64 ? launch_pdl(kv_copy_pages_kernel<64>, grid, dim3(kCopyThreads), 0, st, a)
                                : launch_pdl(kv_copy_pages_kernel<128>, grid, dim3(kCopyThreads), 0, st, a);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

cudaError_t take_pages_flags(unsigned* flags) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_pages_dev_flags, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_pages_dev_flags, &zero, sizeof(zero));
  *flags |= v;
  return e;
}

}  // namespace dustin
