// Verification attention of a batch whose sequences share prefixes: each
// group's prefix is attended to once, by the query rows of all its sequences
// together, beside every sequence's own positions and the window's causal
// block.
//
// Mathematics: softmax over a union of position sets is a weighted mean of
// the sets' softmax outputs, so the work falls into items that are summed
// independently with a running maximum m and sum l per row:
//   prefix item (group, kv head, row tiles)     x the group's prefix tiles,
//   own item    (sequence, kv head, row tiles)  x its own tiles + window's,
// a tile being 128 positions and a row tile 128 of the (sequence, head in
// group, window row) rows that read one kv head.  Items that have two row
// tiles to pair run them side by side over each K/V tile; the odd one runs
// alone, its even and odd K/V tiles side by side.
//
// One persistent CTA per SM; the items' tiles, weighted by row tiles, form
// one line that is cut into equal ranges (lengths are on the device, so every
// CTA computes its cut itself).  Partial results (O unnormalised, m, l) go to
// the workspace, one slot per (CTA, item), and attn_prefix_combine_kernel
// adds each row's partials in a fixed order.
//
// Roles of the 12 warps: 0-3 and 4-7 softmax (one thread per row of stream
// A / B), 8 issues tcgen05.mma, 9 TMA (10 and 11 complete their warpgroup).  S = Q K^T and O += P V accumulate in
// tensor memory (S_A, S_B, O_A, O_B: 512 columns); P replaces S in place as
// bf16 and is read from there as the A operand, so only Q, K and V live in
// shared memory.  While one stream's softmax runs, the tensor cores work on
// the other's products.
#include <algorithm>
#include <cuda.h>

#include "device_common.cuh"
#include "dustin.h"
#include "internal.h"
#include "tcgen05.cuh"

namespace dustin {

namespace {

__device__ unsigned int g_prefix_dev_flags;

constexpr int kTile = 128;        // positions of a K/V tile, rows of a row tile
constexpr int kThreads = 384;
// Registers: a softmax thread holds a row of S (128 values); the producer and
// MMA warps' group gives up what they need beyond the launch's 168.
struct Split {
  static constexpr int NT = kThreads, NPW = 4, NCW = 8;
  static constexpr int PRODUCER_REGS = 72, CONSUMER_REGS = 216;
};
constexpr int kMaskRing = 8;

template <int D>
struct Cfg {
  static constexpr int TILE_BYTES = kTile * D * 2;
  static constexpr int SLOTS = D == 128 ? 5 : 10;
  static constexpr int HALF = kTile * 128;            // bytes of a 64-column half
  static constexpr int SMEM = 1024 + (2 + SLOTS) * TILE_BYTES;
};

// A cache as the kernel sees it; the tensor maps come beside it.
struct PrefixCache {
  const int* page_table;
  int page_size, pages_per_seq, num_pages;
  int box_rows;        // rows of one TMA box
  int zh, zb;          // 0 where that stride is 0: the coordinate stays 0
};

struct PrefixKArgs {
  const __nv_bfloat16* q;
  const int* prefix_len;
  const int* own_len;
  float* ws_o[2];      // partial O: prefix slots, own slots
  float2* ws_ml[2];
  int* plan;           // [0] total, then starts of the groups, of the sequences
  PrefixCache cache[3];
  int n[2];            // prefix, own positions at most
  int count[2];        // groups, sequences
  int row_tiles[2];    // of a prefix, own item family
  int rows[2];         // rows of one (group or sequence, kv head)
  int slot_rows[2];    // rows per stream of a partial slot
  int per, gw, hq_w, hkv, w, win_tiles, grid;
  float scale_log2;
};
struct Maps {
  CUtensorMap k[3], v[3];
};

struct Shared {
  unsigned long long full[10], empty[10];
  unsigned long long q_full[2], s_full[2], p_ready[2], o_final[2], mask_full[kMaskRing], drain;
  unsigned bad[kMaskRing][4];      // positions on pages outside the pool
  int scan[16];
  int start_kind, start_gi, start_pos, total;
  int abort;
  uint32_t tmem;
};

// The clobbers keep a role's set-up code inside the role.
__device__ __forceinline__ void role_begin() { asm volatile("" ::: "memory"); }
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(Split::PRODUCER_REGS) : "memory");
}
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(Split::CONSUMER_REGS) : "memory");
}

__device__ __forceinline__ void raise_flag(unsigned f) { atomicOr(&g_prefix_dev_flags, f); }

// Waits with the library's limit; gives up at once when another role has.
__device__ __forceinline__ bool pwait(unsigned long long* bar, uint32_t parity, int* abort) {
  const uint32_t b = smem_u32(bar);
  if (mbar_try_wait(b, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(b, parity)) {
    if (*(volatile int*)abort || clock64() - t0 > kWaitLimitCycles) {
      *(volatile int*)abort = 1;
      raise_flag(DUSTIN_DEVFLAG_WAIT_TIMEOUT);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool pwait_warp(unsigned long long* bar, uint32_t parity, int* abort) {
  return __all_sync(0xffffffffu, pwait(bar, parity, abort));
}

__device__ __forceinline__ int length_of(const PrefixKArgs& a, int kind, int gi) {
  const int* lens = kind ? a.own_len : a.prefix_len;
  return lens ? min(max(__ldg(lens + gi), 0), a.n[kind]) : a.n[kind];
}
__device__ __forceinline__ int tiles_of(const PrefixKArgs& a, int kind, int len) {
  return (len + kTile - 1) / kTile + (kind ? a.win_tiles : 0);
}
// CTAs that share a line of length total: at least two units each, so that
// every CTA between an item's first and last one has a tile of it (a pair's
// tiles lie two units apart).
__device__ __forceinline__ int sharers(int total, int grid) {
  return max(1, min(grid, total >> 1));
}
// First position of CTA c's range, n CTAs sharing the line.
__device__ __forceinline__ int range_start(int c, int total, int n) {
  return c >= n ? total : (int)(((long long)c * total + n - 1) / n);
}
__device__ __forceinline__ int cta_of(int pos, int total, int n) {
  return (int)((long long)pos * n / total);
}

// One CTA's share of one item.
struct Seg {
  int kind, gi, h, set, item;
  int t0, t1;          // tiles of the item
  int len, hist;       // cached positions, tiles that hold them
  bool pair;
  // Steps of stream s: a pair's streams share every tile, a single's alternate.
  __device__ __forceinline__ int steps(int s) const {
    const int n = t1 - t0;
    return pair ? n : (n + 1 - s) >> 1;
  }
  __device__ __forceinline__ int tile(int s, int step) const {
    return t0 + (pair ? step : 2 * step + s);
  }
  // Ring order of the tiles' K and V (t counted from t0): the order in which
  // the MMA warp is done with them.
  __device__ __forceinline__ int k_at(int t) const { return pair ? 2 * t : t ? 2 * t - 1 : 0; }
  __device__ __forceinline__ int v_at(int t) const {
    return pair ? 2 * t + 1 : t + 1 < t1 - t0 ? 2 * t + 2 : 2 * t + 1;
  }
};

// Walks the segments of [b0, b1); every role walks on its own.
struct Walk {
  const PrefixKArgs& a;
  int b0, b1, kind, gi, h, set, pos, len, tiles;
  __device__ Walk(const PrefixKArgs& args, const Shared& sh) : a(args) {
    const int n = sharers(sh.total, a.grid);
    b0 = range_start(blockIdx.x, sh.total, n);
    b1 = range_start(blockIdx.x + 1, sh.total, n);
    kind = sh.start_kind;
    gi = sh.start_gi;
    pos = sh.start_pos;
    h = set = 0;
    if (b0 >= b1) {
      pos = b1;   // nothing here
    } else {
      load();
      h = (b0 - pos) / (tiles * a.row_tiles[kind]);
      pos += h * tiles * a.row_tiles[kind];
    }
  }
  __device__ __forceinline__ void load() {
    len = length_of(a, kind, gi);
    tiles = tiles_of(a, kind, len);
  }
  __device__ bool next(Seg& s) {
    while (pos < b1) {
      const int rt = a.row_tiles[kind], pairs = rt >> 1;
      if (tiles == 0 || h == a.hkv) {
        h = 0;
        if (++gi == a.count[kind]) {
          gi = 0;
          ++kind;      // pos < b1 <= total: there is work left in kind 1
        }
        load();
        continue;
      }
      const bool pair = set < pairs;
      const int wt = pair ? 2 : 1;
      const int lo = b0 > pos ? (b0 - pos + wt - 1) / wt : 0;
      const int hi = min(tiles, (b1 - pos + wt - 1) / wt);
      s.kind = kind;
      s.gi = gi;
      s.h = h;
      s.set = set;
      s.item = (gi * a.hkv + h) * ((rt + 1) >> 1) + set;
      s.t0 = lo;
      s.t1 = hi;
      s.len = len;
      s.hist = (len + kTile - 1) / kTile;
      s.pair = pair;
      pos += tiles * wt;
      if (++set == (rt + 1) >> 1) {
        set = 0;
        ++h;
      }
      if (lo < hi) return true;
    }
    return false;
  }
};

// The line's length, where this CTA's range starts, and (CTA 0) the starts of
// all groups and sequences for the combine kernel.
__device__ void make_plan(const PrefixKArgs& a, Shared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int base = 0, first[2];
  int mine_lo[2], mine_hi[2];
  for (int kind = 0; kind < 2; ++kind) {
    const int unit = a.hkv * a.row_tiles[kind];
    const int m = (a.count[kind] + kThreads - 1) / kThreads;
    const int lo = min(tid * m, a.count[kind]), hi = min(lo + m, a.count[kind]);
    int sum = 0;
    for (int i = lo; i < hi; ++i) sum += tiles_of(a, kind, length_of(a, kind, i)) * unit;
    int inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += y;
    }
    __syncthreads();
    if (lane == 31) sh.scan[warp] = inc;
    __syncthreads();
    int below = 0, all = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) below += sh.scan[i];
      all += sh.scan[i];
    }
    first[kind] = base + below + inc - sum;
    mine_lo[kind] = lo;
    mine_hi[kind] = hi;
    base += all;
  }
  const int total = base;
  if (tid == 0) {
    sh.total = total;
    if (blockIdx.x == 0) a.plan[0] = total;
  }
  const int b0 = range_start(blockIdx.x, total, sharers(total, a.grid));
  for (int kind = 0; kind < 2; ++kind) {
    const int unit = a.hkv * a.row_tiles[kind];
    int at = first[kind];
    for (int i = mine_lo[kind]; i < mine_hi[kind]; ++i) {
      const int next = at + tiles_of(a, kind, length_of(a, kind, i)) * unit;
      if (at <= b0 && b0 < next) {
        sh.start_kind = kind;
        sh.start_gi = i;
        sh.start_pos = at;
      }
      if (blockIdx.x == 0) a.plan[1 + kind * a.count[0] + i] = at;
      at = next;
    }
  }
  __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prefix_kernel(const __grid_constant__ PrefixKArgs a, const __grid_constant__ Maps maps) {
  using C = Cfg<D>;
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t q_buf = base, ring = base + 2 * C::TILE_BYTES;

  if (tid == 0) {
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sh.q_full[s]), 4);
      mbar_init(smem_u32(&sh.s_full[s]), 1);
      mbar_init(smem_u32(&sh.p_ready[s]), 4);
      mbar_init(smem_u32(&sh.o_final[s]), 1);
    }
    for (int i = 0; i < kMaskRing; ++i) mbar_init(smem_u32(&sh.mask_full[i]), 1);
    mbar_init(smem_u32(&sh.drain), 1);
    mbar_fence_init();
    sh.abort = 0;
  }
  if (warp == 8) tmem_alloc<512>(smem_u32(&sh.tmem));
  griddep_wait();
  griddep_launch_dependents();
  make_plan(a, sh);          // ends with a CTA barrier
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  if (warp >= 8) give_registers();   // one instruction for the whole warpgroup
  if (warp == 9) {
    // ------------------------------------------------------------- producer
    role_begin();
    Walk walk(a, sh);
    Seg s;
    int slot = 0, tile_count = 0;
    uint32_t phase = 0;
    int filled = 0;          // slots filled at least once
    bool ok = true;
    while (ok && walk.next(s)) {
      const int n = s.t1 - s.t0;
      int kt = 0, vt = 0;    // next K, V tile
      for (int x = 0; ok && x < 2 * n; ++x) {
        const bool is_k = kt < n && s.k_at(kt) == x;
        const int t = s.t0 + (is_k ? kt++ : vt++);
        ok = pwait_warp(&sh.empty[slot], phase ^ 1, &sh.abort);
        if (!ok) break;
        const uint32_t bar = smem_u32(&sh.full[slot]);
        const uint32_t dst = ring + slot * C::TILE_BYTES;
        const bool window = s.kind && t >= s.hist;
        const int ci = window ? 2 : s.kind;
        const PrefixCache& c = a.cache[ci];
        const CUtensorMap* map = is_k ? &maps.k[ci] : &maps.v[ci];
        const int row0 = (window ? t - s.hist : t) * kTile;
        if (lane == 0) mbar_arrive_expect_tx(bar, C::TILE_BYTES);
        if (!c.page_table) {
          __syncwarp();
          if (lane < D / 64)
            tma_load_4d(dst + lane * C::HALF, map, lane * 64, row0, s.h * c.zh, s.gi * c.zb, bar);
        } else {
          // One box per (run of box_rows positions, 64-column half); a run
          // lies on one page.  Pages behind the end or outside the pool load
          // as zeros (a coordinate past the map's extent).
          unsigned bad = 0;
          const int boxes = kTile / c.box_rows;
          int page = c.num_pages, r = 0;
          if (lane < boxes * (D / 64)) {
            r = lane % boxes * c.box_rows;
            const int j = row0 + r;
            if (j < s.len) {
              page = __ldg(c.page_table + (long long)s.gi * c.pages_per_seq + j / c.page_size);
              if (page < 0 || page >= c.num_pages) {
                page = c.num_pages;
                bad = 1;
                raise_flag(DUSTIN_DEVFLAG_PAGE_RANGE);
              } else {
                page *= c.zb;
              }
            }
          }
          if (is_k) {
            // Positions on bad pages, for the softmax.
            const unsigned runs = __ballot_sync(0xffffffffu, bad != 0);
            if (lane < 4) {
              unsigned bits = 0;
              for (int i = 0; i < 32; ++i)
                if (runs >> ((lane * 32 + i) / c.box_rows) & 1) bits |= 1u << i;
              sh.bad[tile_count % kMaskRing][lane] = runs ? bits : 0;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.mask_full[tile_count % kMaskRing]));
          }
          __syncwarp();
          if (lane < boxes * (D / 64)) {
            const int half = lane / boxes;
            tma_load_4d(dst + half * C::HALF + r * 128, map, half * 64,
                        (row0 + r) % c.page_size, s.h * c.zh, page, bar);
          }
        }
        if (is_k && c.page_table) ++tile_count;
        filled = min(filled + 1, C::SLOTS);
        if (++slot == C::SLOTS) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    // Given up: the copies in flight land before the CTA's memory is reused.
    if (!ok) {
      for (int i = 0; i < filled; ++i) {
        slot = slot == 0 ? C::SLOTS - 1 : slot - 1;
        if (slot == C::SLOTS - 1) phase ^= 1;
        mbar_wait(smem_u32(&sh.full[slot]), phase, kWaitLimitCycles);
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------------ MMA
    role_begin();
    if (lane == 0) {
      Walk walk(a, sh);
      Seg s;
      constexpr uint32_t kQk = mma_idesc(128, 128, false), kPv = mma_idesc(128, D, true);
      int ring0 = 0;                        // ring position of the segment's first slot
      uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
      bool ok = true;
      auto full = [&](int at) {
        return pwait(&sh.full[at % C::SLOTS], (at / C::SLOTS) & 1, &sh.abort);
      };
      auto qk = [&](int st, int at) {
        const uint64_t qd = smem_desc(q_buf + st * C::TILE_BYTES, 16, 1024);
        const uint64_t kd = smem_desc(ring + at % C::SLOTS * C::TILE_BYTES, 16, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (uint32_t)((k / 4) * C::HALF + (k % 4) * 32) >> 4;
          mma_ss(tmem + st * 128, qd + off, kd + off, kQk, k > 0);
        }
        mma_commit(smem_u32(&sh.s_full[st]));
      };
      auto pv = [&](int st, int at, bool acc) {
        const uint64_t vd = smem_desc(ring + at % C::SLOTS * C::TILE_BYTES, C::HALF, 1024);
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_ts(tmem + 256 + st * 128, tmem + st * 128 + k * 8, vd + (uint32_t)(k * 2048 >> 4),
                 kPv, acc || k > 0);
      };
      auto release = [&](int at) { mma_commit(smem_u32(&sh.empty[at % C::SLOTS])); };
      while (ok && walk.next(s)) {
        const int last = s.pair ? 1 : 0;   // the stream after which a pair's slot is free
        for (int st = 0; ok && st < 2; ++st) {
          if (s.steps(st) == 0) continue;
          const int at = ring0 + s.k_at(s.tile(st, 0) - s.t0);
          ok = pwait(&sh.q_full[st], q_phase[st], &sh.abort) && full(at);
          if (!ok) break;
          q_phase[st] ^= 1;
          tc_fence_after();
          qk(st, at);
          if (!s.pair || st == last) release(at);
        }
        for (int step = 0; ok && step < s.steps(0); ++step) {
          for (int st = 0; ok && st < 2; ++st) {
            if (step >= s.steps(st)) continue;
            const int vat = ring0 + s.v_at(s.tile(st, step) - s.t0);
            ok = pwait(&sh.p_ready[st], p_phase[st], &sh.abort) && full(vat);
            if (!ok) break;
            p_phase[st] ^= 1;
            tc_fence_after();
            pv(st, vat, step > 0);
            if (!s.pair || st == last) release(vat);
            if (step + 1 < s.steps(st)) {
              const int kat = ring0 + s.k_at(s.tile(st, step + 1) - s.t0);
              ok = full(kat);
              if (!ok) break;
              qk(st, kat);
              if (!s.pair || st == last) release(kat);
            } else {
              mma_commit(smem_u32(&sh.o_final[st]));
            }
          }
        }
        ring0 += 2 * (s.t1 - s.t0);
      }
      if (!ok) {   // given up: the products in flight end before tensor memory is freed
        mma_commit(smem_u32(&sh.drain));
        mbar_wait(smem_u32(&sh.drain), 0, kWaitLimitCycles);
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    // -------------------------------------------------------------- softmax
    take_registers();
    const int st = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // TMEM lane of the warp's first row
    const uint32_t tS = tmem + lanes + st * 128, tO = tmem + lanes + 256 + st * 128;
    Walk walk(a, sh);
    Seg s;
    int ring0 = 0, tile_count = 0;
    uint32_t s_phase = 0, o_phase = 0;
    bool ok = true;
    while (ok && walk.next(s)) {
      const int steps = s.steps(st);
      const int rt = s.pair ? 2 * s.set + st : 2 * (a.row_tiles[s.kind] >> 1);
      const int rows = min(kTile, a.rows[s.kind] - rt * kTile);
      const long long slot = (long long)(blockIdx.x + s.item) * 2 + st;
      float2* ml = a.ws_ml[s.kind] + slot * a.slot_rows[s.kind];
      const int paged_tiles0 = tile_count;
      if (a.cache[s.kind].page_table)
        tile_count += max(0, min(s.t1, s.hist) - s.t0);
      if (steps == 0) {
        if (row < rows) ml[row] = make_float2(-INFINITY, 0.f);
        ring0 += 2 * (s.t1 - s.t0);
        continue;
      }
      // Q rows, swizzled as the tensor cores read them; absent rows are zero.
      {
        constexpr int CPR = D / 8;
        const uint32_t dst = q_buf + st * C::TILE_BYTES;
#pragma unroll 4
        for (int i = row; i < kTile * CPR; i += 128) {
          const int r = i / CPR, c = i % CPR;
          const int rr = rt * kTile + r;
          const int seq = s.kind ? s.gi : s.gi * a.per + rr / a.gw;
          const int in_seq = s.kind ? rr : rr % a.gw;
          const bool have = r < rows;
          const __nv_bfloat16* src =
              a.q + (have ? ((long long)seq * a.hq_w + s.h * a.gw + in_seq) * D + c * 8 : 0);
          cp_async_16(dst + (c / 8) * C::HALF + r * 128 + ((c % 8 ^ (r & 7)) << 4), src,
                      have ? 16 : 0);
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.q_full[st]));
      }
      const bool live = (warp & 3) * 32 < rows;           // the warp has rows
      int t_row = 0;                                      // window row of this row
      if (s.kind) t_row = (rt * kTile + row) % a.w;
      float m = -INFINITY, l = 0.f;
      for (int step = 0; step < steps; ++step) {
        const int t = s.tile(st, step);
        ok = pwait_warp(&sh.s_full[st], s_phase, &sh.abort);
        if (!ok) break;
        s_phase ^= 1;
        tc_fence_after();
        // Columns [0, lim) count.
        int lim;
        const bool window = s.kind && t >= s.hist;
        if (window)
          lim = min(a.w, t_row + 1) - (t - s.hist) * kTile;
        else
          lim = s.len - t * kTile;
        const bool paged = !window && a.cache[s.kind].page_table;
        const int mslot = (paged_tiles0 + t - s.t0) % kMaskRing;
        if (paged) {
          ok = pwait_warp(&sh.mask_full[mslot],
                          ((paged_tiles0 + t - s.t0) / kMaskRing) & 1, &sh.abort);
          if (!ok) break;
        }
        if (live) {
          uint32_t x[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, x[c]);
          tc_wait_ld();
          if (__any_sync(0xffffffffu, lim < kTile)) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (c * 32 + i >= lim) x[c][i] = 0xff800000u;   // -inf
          }
          if (paged) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const unsigned bad = sh.bad[mslot][c];
              if (bad) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (bad >> i & 1) x[c][i] = 0xff800000u;
              }
            }
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            mx[c] = __uint_as_float(x[c][0]);
#pragma unroll
            for (int i = 1; i < 32; ++i) mx[c] = fmaxf(mx[c], __uint_as_float(x[c][i]));
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
          // The reference maximum moves only when a tile exceeds it by more
          // than a factor 2^8 (or sets it): P stays below 2^8, and O is
          // rescaled a few times per item.
          const bool up = top > m + kLazyRescale || (m == -INFINITY && top > m);
          if (__any_sync(0xffffffffu, up)) {
            const float m_new = up ? top : m;
            const float f = up ? ex2(m - m_new) : 1.f;
            m = m_new;
            l *= f;
            if (step > 0) {
              // The product that wrote O was issued before the one that
              // signalled S: it is complete.
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tO + c * 32, o);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st32(tO + c * 32, o);
              }
            }
          }
          const float ms = m == -INFINITY ? 0.f : m;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float e0 = ex2(fmaf(__uint_as_float(x[c][2 * i]), a.scale_log2, -ms));
              const float e1 = ex2(fmaf(__uint_as_float(x[c][2 * i + 1]), a.scale_log2, -ms));
              sum[i & 3] += e0 + e1;
              // P in bf16, as the tensor cores take it (relative rounding
              // 2^-8 per weight); the row sum keeps the fp32 values.
              p[i] = pack_bf16(e0, e1);
            }
            tmem_st16(tS + c * 16, p);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tc_wait_st();
        }
        // V rows behind the end hold whatever the cache holds there, NaN
        // included: 0 * NaN must not reach O.
        const int valid = s.len - t * kTile;
        if (!window && valid < kTile && (!s.pair || st == 0)) {
          const int vat = ring0 + s.v_at(t - s.t0);
          ok = pwait_warp(&sh.full[vat % C::SLOTS], (vat / C::SLOTS) & 1, &sh.abort);
          if (!ok) break;
          const uint32_t v = ring + vat % C::SLOTS * C::TILE_BYTES;
          for (int i = valid * 8 + row; i < kTile * 8; i += 128)
#pragma unroll
            for (int half = 0; half < D / 64; ++half)
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};\n" ::"r"(
                               v + half * C::HALF + i * 16),
                           "r"(0)
                           : "memory");
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.p_ready[st]));
      }
      if (!ok) break;
      ok = pwait_warp(&sh.o_final[st], o_phase, &sh.abort);
      if (!ok) break;
      o_phase ^= 1;
      tc_fence_after();
      if (live) {
        float* out = a.ws_o[s.kind] + (slot * a.slot_rows[s.kind] + row) * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + c * 32, o);
          tc_wait_ld();
          if (row < rows) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4*>(out + c * 32 + i) =
                  make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
        if (row < rows) ml[row] = make_float2(m, l);
      }
      ring0 += 2 * (s.t1 - s.t0);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc<512>(tmem);
}

// ---- combine: one warp per output row

struct CombineArgs {
  PrefixKArgs k;
  __nv_bfloat16* o;
  float* lse;
  long long rows;      // b * h_q * w
};

constexpr int kCombineWarps = 8;

template <int D>
__global__ void __launch_bounds__(kCombineWarps * 32)
    attn_prefix_combine_kernel(const __grid_constant__ CombineArgs c) {
  constexpr int CPL = D / 32;
  const PrefixKArgs& a = c.k;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kCombineWarps + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  if (row >= c.rows) return;
  const int seq = (int)(row / a.hq_w), in_seq = (int)(row % a.hq_w);
  const int h = in_seq / a.gw, r = in_seq % a.gw;
  const int total = a.plan[0], n_cta = sharers(total, a.grid);
  // Partials of the row: parts[0] of its prefix item, then parts[1] of its own.
  int parts[2], first_cta[2], item[2], in_tile[2], twice[2], stream[2];
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const int gi = kind ? seq : seq / a.per;
    const int rr = kind ? r : seq % a.per * a.gw + r;
    const int rt = rr / kTile, pairs = a.row_tiles[kind] >> 1, set = rt >> 1;
    const bool pair = set < pairs;
    const int tiles = a.count[kind] ? tiles_of(a, kind, length_of(a, kind, gi)) : 0;
    parts[kind] = 0;
    in_tile[kind] = rr % kTile;
    stream[kind] = pair ? rt & 1 : 0;
    twice[kind] = pair ? 0 : 1;
    item[kind] = (gi * a.hkv + h) * ((a.row_tiles[kind] + 1) >> 1) + set;
    first_cta[kind] = 0;
    if (tiles > 0) {
      const int start = a.plan[1 + kind * a.count[0] + gi] +
                        (h * a.row_tiles[kind] + set * 2) * tiles;
      first_cta[kind] = cta_of(start, total, n_cta);
      const int last = cta_of(start + (tiles - 1) * (pair ? 2 : 1), total, n_cta);
      parts[kind] = (last - first_cta[kind] + 1) << twice[kind];
    }
  }
  const int n = parts[0] + parts[1];
  // Row index (in rows of its workspace) of partial i.
  auto where = [&](int i, int& kind) {
    kind = i >= parts[0];
    const int x = kind ? i - parts[0] : i;
    const int cta = first_cta[kind] + (x >> twice[kind]);
    const int st = twice[kind] ? x & 1 : stream[kind];
    return ((long long)(cta + item[kind]) * 2 + st) * a.slot_rows[kind] + in_tile[kind];
  };
  float top = -INFINITY;
  for (int i = lane; i < n; i += 32) {
    int kind;
    const long long at = where(i, kind);
    top = fmaxf(top, a.ws_ml[kind][at].x);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  const float m = top == -INFINITY ? 0.f : top;
  float acc[CPL] = {};
  float l = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    float weight = 0.f, lsum = 0.f;
    long long at = 0;
    int kind = 0;
    if (i0 + lane < n) {
      at = where(i0 + lane, kind);
      const float2 ml = a.ws_ml[kind][at];
      weight = ex2(ml.x - m);
      lsum = ml.y * weight;
    }
    l += lsum;
    const int count = min(32, n - i0);
#pragma unroll 4
    for (int i = 0; i < count; ++i) {
      const float wi = __shfl_sync(0xffffffffu, weight, i);
      const long long ai = __shfl_sync(0xffffffffu, at, i);
      const int ki = __shfl_sync(0xffffffffu, kind, i);
      if (wi == 0.f) continue;   // nothing seen there (O may be unwritten)
      const float* src = a.ws_o[ki] + ai * D + lane * CPL;
      float v[CPL];
      if constexpr (CPL == 4) {
        const float4 f = *reinterpret_cast<const float4*>(src);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(src);
        v[0] = f.x, v[1] = f.y;
      }
#pragma unroll
      for (int x = 0; x < CPL; ++x) acc[x] = fmaf(wi, v[x], acc[x]);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  const float inv = top == -INFINITY ? 0.f : 1.f / l;
  uint32_t out[CPL / 2];
#pragma unroll
  for (int x = 0; x < CPL / 2; ++x) out[x] = pack_bf16(acc[2 * x] * inv, acc[2 * x + 1] * inv);
  __nv_bfloat16* dst = c.o + row * D + lane * CPL;
  if constexpr (CPL == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  else
    *reinterpret_cast<uint32_t*>(dst) = out[0];
  if (lane == 0) c.lse[row] = top == -INFINITY ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ---- host side

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
  static std::atomic<EncodeTiledFn> fn{nullptr};
  EncodeTiledFn f = fn.load(std::memory_order_acquire);
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                       &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess && p) {
    f = reinterpret_cast<EncodeTiledFn>(p);
    fn.store(f, std::memory_order_release);
  }
  return f;
}

// [outer][h_kv][rows][d] of one cache tensor as 64-column boxes.  An axis of
// stride 0 becomes an axis of one element.
bool make_map(CUtensorMap* map, const __nv_bfloat16* base, int d, long long rows, long long heads,
              long long outer, const KvView& kv, int box_rows) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)rows,
                              (cuuint64_t)(kv.sh ? heads : 1), (cuuint64_t)(kv.sb ? outer : 1)};
  const cuuint64_t strides[3] = {(cuuint64_t)kv.sn * 2, (cuuint64_t)(kv.sh ? kv.sh : kv.sn) * 2,
                                 (cuuint64_t)(kv.sb ? kv.sb : kv.sn) * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<__nv_bfloat16*>(base), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Layout {
  size_t o[2], ml[2], plan, total;
};

// Sizes that depend on the shape alone (not on the lengths).
PrefixKArgs shape_args(const PrefixArgs& p, int sms, Layout* lay) {
  PrefixKArgs a{};
  a.per = p.b / p.groups;
  a.gw = p.hq / p.hkv * p.w;
  a.hq_w = p.hq * p.w;
  a.hkv = p.hkv;
  a.w = p.w;
  a.n[0] = p.n_prefix;
  a.n[1] = p.n_own;
  a.count[0] = p.groups;
  a.count[1] = p.b;
  a.rows[0] = a.per * a.gw;
  a.rows[1] = a.gw;
  for (int k = 0; k < 2; ++k) {
    a.row_tiles[k] = (a.rows[k] + kTile - 1) / kTile;
    a.slot_rows[k] = std::min(kTile, a.rows[k]);
  }
  // The workspace does not depend on whether the window comes along.
  a.win_tiles = (p.w + kTile - 1) / kTile;
  a.grid = sms;
  size_t at = 0;
  for (int k = 0; k < 2; ++k) {
    const size_t items = (size_t)a.count[k] * a.hkv * ((a.row_tiles[k] + 1) / 2);
    const size_t rows = (items + a.grid) * 2 * a.slot_rows[k];
    lay->o[k] = at;
    at += align256(rows * p.d * sizeof(float));
    lay->ml[k] = at;
    at += align256(rows * sizeof(float2));
  }
  lay->plan = at;
  at += align256((size_t)(1 + p.groups + p.b) * sizeof(int));
  lay->total = at;
  return a;
}

template <int D>
cudaError_t run_prefix(const PrefixKArgs& k, const Maps& maps, const PrefixArgs& p,
                       cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  auto kern = attn_prefix_kernel<D>;
  cudaError_t e = ensure_smem_attr(kern, Cfg<D>::SMEM, done);
  if (e != cudaSuccess) return e;
  static std::atomic<int> split_ok{0};
  if ((e = check_register_split<Split>(kern, split_ok)) != cudaSuccess) return e;
  e = launch_pdl(kern, dim3((unsigned)k.grid), dim3(kThreads), Cfg<D>::SMEM, st, k, maps);
  if (e != cudaSuccess) return e;
  note_launches(1);
  CombineArgs c{};
  c.k = k;
  c.o = p.o;
  c.lse = p.lse;
  c.rows = (long long)p.b * p.hq * p.w;
  e = launch_pdl(attn_prefix_combine_kernel<D>,
                 dim3((unsigned)((c.rows + kCombineWarps - 1) / kCombineWarps)),
                 dim3(kCombineWarps * 32), 0, st, c);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace

size_t prefix_workspace(const PrefixArgs& p, int sms) {
  Layout lay;
  shape_args(p, sms, &lay);
  return lay.total;
}

cudaError_t launch_attn_prefix(const PrefixArgs& p, int sms, void* ws, cudaStream_t st) {
  Layout lay;
  PrefixKArgs a = shape_args(p, sms, &lay);
  if (!p.has_win) a.win_tiles = 0;
  a.q = p.q;
  a.prefix_len = p.prefix_len;
  a.own_len = p.own_len;
  a.scale_log2 = p.scale_log2;
  char* base = static_cast<char*>(ws);
  for (int k = 0; k < 2; ++k) {
    a.ws_o[k] = reinterpret_cast<float*>(base + lay.o[k]);
    a.ws_ml[k] = reinterpret_cast<float2*>(base + lay.ml[k]);
  }
  a.plan = reinterpret_cast<int*>(base + lay.plan);
  Maps maps;
  const KvView* views[3] = {p.n_prefix > 0 ? &p.prefix : nullptr, p.n_own > 0 ? &p.own : nullptr,
                            p.has_win ? &p.win : nullptr};
  const int rows[3] = {p.n_prefix, p.n_own, p.w};
  for (int c = 0; c < 3; ++c) {
    if (!views[c]) continue;
    const KvView& kv = *views[c];
    PrefixCache& pc = a.cache[c];
    const bool paged = kv.page_table != nullptr;
    pc.page_table = kv.page_table;
    pc.page_size = kv.page_size;
    pc.pages_per_seq = kv.pages_per_seq;
    pc.num_pages = kv.num_pages;
    pc.box_rows = kTile;
    if (paged)   // the largest power of two that divides the page and the tile
      for (pc.box_rows = 16; pc.box_rows < kTile && kv.page_size % (2 * pc.box_rows) == 0;)
        pc.box_rows *= 2;
    pc.zh = kv.sh ? 1 : 0;
    pc.zb = kv.sb ? 1 : 0;
    const long long outer = paged ? kv.num_pages : c == 0 ? p.groups : p.b;
    const long long r = paged ? kv.page_size : rows[c];
    if (!make_map(&maps.k[c], kv.k, p.d, r, p.hkv, outer, kv, pc.box_rows) ||
        !make_map(&maps.v[c], kv.v, p.d, r, p.hkv, outer, kv, pc.box_rows))
      return cudaErrorNotSupported;
  }
  return p.d == 64 ? run_prefix<64>(a, maps, p, st) : run_prefix<128>(a, maps, p, st);
}

cudaError_t take_prefix_flags(unsigned* flags) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_prefix_dev_flags, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_prefix_dev_flags, &zero, sizeof(zero));
  *flags |= v;
  return e;
}

}  // namespace dustin
