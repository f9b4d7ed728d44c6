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
// Roles of the 20 warps: 0-7 and 8-15 softmax of stream A / B (two threads
// per row, 64 columns each), 16 issues tcgen05.mma, 17 TMA loads of K and V,
// 18 copies Q rows, 19 walks the CTA's range and publishes its segments.
// S = Q K^T and O += P V accumulate in tensor memory (S_A, S_B, O_A, O_B:
// 512 columns); P replaces S in place as bf16 and is read from there as the A
// operand, so only Q, K and V live in shared memory.  While one stream's
// softmax runs, the tensor cores work on the other's products.
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
constexpr int kSoftmaxWarps = 8;  // per stream
constexpr int kThreads = (2 * kSoftmaxWarps + 4) * 32;
// Registers: a softmax thread holds half a row of S (64 values); the other
// warpgroup gives up what they need beyond the launch's 96.
struct Split {
  static constexpr int NT = kThreads, NPW = 4, NCW = 2 * kSoftmaxWarps;
  static constexpr int PRODUCER_REGS = 64, CONSUMER_REGS = 104;
};
constexpr int kMaskRing = 8;
constexpr int kSegRing = 4;

template <int D>
struct Cfg {
  static constexpr int TILE_BYTES = kTile * D * 2;
  static constexpr int SLOTS = D == 128 ? 5 : 10;
  static constexpr int HALF = kTile * 128;            // bytes of a 64-column half
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

// One CTA's share of one item.
struct Seg {
  int kind;            // 0 prefix, 1 own, -1: no more
  int gi, h, rt;       // group or sequence, kv head, first row tile
  int t0, n;           // tiles of the item
  int len, hist;       // cached positions, tiles that hold them
  int slot;            // partial slot
  int pair;
  // Steps of stream s: a pair's streams share every tile, a single's alternate.
  __device__ __forceinline__ int steps(int s) const { return pair ? n : (n + 1 - s) >> 1; }
  // Tile of a step, counted from t0.
  __device__ __forceinline__ int tile(int s, int step) const { return pair ? step : 2 * step + s; }
  // Ring order of the tiles' K and V: the order in which the MMA warp is
  // done with them.
  __device__ __forceinline__ int k_at(int t) const { return pair ? 2 * t : t ? 2 * t - 1 : 0; }
  __device__ __forceinline__ int v_at(int t) const {
    return pair ? 2 * t + 1 : t + 1 < n ? 2 * t + 2 : 2 * t + 1;
  }
};

struct Control {
  float exchange[2][2][kTile];     // between the two threads of a row
  unsigned long long full[10], empty[10];
  unsigned long long q_full[2], q_empty[2], s_full[2], p_ready[2], o_final[2];
  unsigned long long seg_full[kSegRing], seg_empty[kSegRing], mask_full[kMaskRing], drain;
  unsigned bad[kMaskRing][4];      // positions on pages outside the pool
  Seg seg[kSegRing];
  int abort;
  uint32_t tmem;
};

template <int D>
constexpr int kSmem = (2 + Cfg<D>::SLOTS) * Cfg<D>::TILE_BYTES + (int)sizeof(Control);
static_assert(kSmem<128> <= 232448, "shared memory of one CTA");

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
// The line cut into n ranges: range c starts at ceil(c * total / n), which is
// c * (total / n) + ceil(c * (total % n) / n), all in 32 bits.
struct Cut {
  int n, total, q, r;
  __device__ __forceinline__ Cut(int line, int grid) {
    total = line;
    n = sharers(line, grid);
    q = total / n;
    r = total - q * n;
  }
  __device__ __forceinline__ int start(int c) const {
    return c >= n ? total : c * q + (c * r + n - 1) / n;
  }
  // The range that holds pos: a float estimate, at most one off, put right.
  __device__ __forceinline__ int of(int pos) const {
    int c = min((int)((float)pos * (float)n / (float)total), n - 1);
    while (start(c) > pos) --c;
    while (start(c + 1) <= pos) ++c;
    return c;
  }
};

// Walks the segments of [b0, b1).
struct Walk {
  const PrefixKArgs& a;
  int b0, b1, kind, gi, h, set, pos, len, tiles;
  __device__ explicit Walk(const PrefixKArgs& args) : a(args) {
    plan();
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
  // The range [b0, b1) and the group or sequence it starts in; CTA 0 leaves
  // the line's length and all starts on it for the combine kernel.  A warp
  // scans the lengths, 32 at a time, twice (for the length, for the start).
  __device__ void plan() {
    const int lane = threadIdx.x & 31;
    int total = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      int sum = 0;
      if ((k ? a.own_len : a.prefix_len) == nullptr) {
        sum = a.count[k] * tiles_of(a, k, a.n[k]);
      } else {
        for (int i = lane; i < a.count[k]; i += 32) sum += tiles_of(a, k, length_of(a, k, i));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      }
      total += sum * a.hkv * a.row_tiles[k];
    }
    const Cut cut(total, a.grid);
    b0 = cut.start(blockIdx.x);
    b1 = cut.start(blockIdx.x + 1);
    kind = gi = pos = 0;
    int base = 0;
    if (blockIdx.x == 0 && lane == 0) a.plan[0] = total;
    for (int k = 0; k < 2; ++k) {
      const int unit = a.hkv * a.row_tiles[k];
      for (int i0 = 0; i0 < a.count[k]; i0 += 32) {
        const int i = i0 + lane;
        const int mine = i < a.count[k] ? tiles_of(a, k, length_of(a, k, i)) * unit : 0;
        int inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, d);
          if (lane >= d) inc += y;
        }
        const int at = base + inc - mine;
        if (blockIdx.x == 0 && i < a.count[k]) a.plan[1 + k * a.count[0] + i] = at;
        const unsigned here = __ballot_sync(0xffffffffu, at <= b0 && b0 < at + mine);
        if (here) {
          const int src = __ffs((int)here) - 1;
          kind = k;
          gi = i0 + src;
          pos = __shfl_sync(0xffffffffu, at, src);
          if (blockIdx.x != 0) return;
        }
        base += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
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
      s.rt = 2 * set;
      s.slot = blockIdx.x + (gi * a.hkv + h) * ((rt + 1) >> 1) + set;
      s.t0 = lo;
      s.n = hi - lo;
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

// ---- softmax arithmetic: two columns at a time

__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
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
__device__ __forceinline__ float max32(const uint32_t (&x)[32], float top) {
  float a = top, b = __uint_as_float(x[0]);
#pragma unroll
  for (int i = 1; i < 29; i += 4) {
    a = max3(a, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
    b = max3(b, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
  }
  a = max3(a, __uint_as_float(x[29]), __uint_as_float(x[30]));
  return max3(a, b, __uint_as_float(x[31]));
}
// p = 2^(x * scale - m) as 16 bf16 pairs, the fp32 values added to sum, the
// largest x to top.
__device__ __forceinline__ void exp32(const uint32_t (&x)[32], uint64_t scale, uint64_t minus_m,
                                      uint64_t (&sum)[2], float& top, uint32_t* p) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    top = max3(top, __uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
    const uint64_t y = fma2(pack2(x[2 * i], x[2 * i + 1]), scale, minus_m);
    const float e0 = ex2(lo_of(y)), e1 = ex2(hi_of(y));
    sum[i & 1] = add2(sum[i & 1], pack2(__float_as_uint(e0), __float_as_uint(e1)));
    // P in bf16, as the tensor cores take it (relative rounding 2^-8 per
    // weight); the row sum keeps the fp32 values.
    p[i] = pack_bf16(e0, e1);
  }
}
// Columns [lim, 32) of x do not count.
__device__ __forceinline__ void mask32(uint32_t (&x)[32], int lim) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i >= lim) x[i] = 0xff800000u;   // -inf
}
__device__ __forceinline__ void mask_bits(uint32_t (&x)[32], unsigned bad) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (bad >> i & 1) x[i] = 0xff800000u;
}

// Barrier of the two warps that share 32 rows; whether any thread said yes.
__device__ __forceinline__ bool pair_any(int id, bool yes) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " bar.red.or.pred q, %2, 64, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)yes), "r"(id)
      : "memory");
  return r != 0;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prefix_kernel(const __grid_constant__ PrefixKArgs a, const __grid_constant__ Maps maps) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) unsigned char raw[];
  Control& sh = *reinterpret_cast<Control*>(raw + (2 + C::SLOTS) * C::TILE_BYTES);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t q_buf = smem_u32(raw), ring = q_buf + 2 * C::TILE_BYTES;

  if (tid == 0) {
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sh.q_full[s]), 1);
      mbar_init(smem_u32(&sh.q_empty[s]), 1);
      mbar_init(smem_u32(&sh.s_full[s]), 1);
      mbar_init(smem_u32(&sh.p_ready[s]), kSoftmaxWarps);
      mbar_init(smem_u32(&sh.o_final[s]), 1);
    }
    for (int i = 0; i < kMaskRing; ++i) mbar_init(smem_u32(&sh.mask_full[i]), 1);
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(smem_u32(&sh.seg_full[i]), 1);
      mbar_init(smem_u32(&sh.seg_empty[i]), 2 * kSoftmaxWarps + 3);
    }
    mbar_init(smem_u32(&sh.drain), 1);
    mbar_fence_init();
    sh.abort = 0;
  }
  if (warp == 16) tmem_alloc<512>(smem_u32(&sh.tmem));
  // Rows a row tile lacks keep finite values: zeros, later another tile's.
  for (int i = tid; i < 2 * C::TILE_BYTES / 16; i += kThreads)
    *reinterpret_cast<uint4*>(raw + i * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tmem = sh.tmem;

  // Segment `at` of the ring, once published; null: given up.
  auto segment = [&](int at) -> const Seg* {
    if (!pwait_warp(&sh.seg_full[at % kSegRing], (at / kSegRing) & 1, &sh.abort)) return nullptr;
    return &sh.seg[at % kSegRing];
  };
  auto done_with = [&](int at) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.seg_empty[at % kSegRing]));
  };

  if (warp >= 16) give_registers();   // one instruction for the whole warpgroup
  if (warp == 19) {
    // --------------------------------------------------------------- walker
    role_begin();
    Walk walk(a);
    Seg s;
    for (int at = 0;; ++at) {
      const bool more = walk.next(s);
      if (!pwait_warp(&sh.seg_empty[at % kSegRing], (at / kSegRing & 1) ^ 1, &sh.abort)) break;
      if (!more) s.kind = -1;
      if (lane == 0) {
        sh.seg[at % kSegRing] = s;
        mbar_arrive(smem_u32(&sh.seg_full[at % kSegRing]));
      }
      if (!more) break;
    }
  } else if (warp == 18) {
    // ------------------------------------------------------------------- Q
    // Row tiles in the tensor cores' swizzled layout; a pair fills both
    // buffers, singles take turns, so that the next one's rows are there
    // before this one ends.
    role_begin();
    int fills[2] = {0, 0}, turn = 0;
    for (int at = 0;; ++at) {
      const Seg* sp = segment(at);
      if (!sp || sp->kind < 0) break;
      const Seg s = *sp;
      done_with(at);
      bool ok = true;
      for (int i = 0; ok && i <= s.pair; ++i) {
        const int buf = s.pair ? i : turn;
        const int first = (s.rt + i) * kTile;
        const int rows = min(kTile, a.rows[s.kind] - first);
        ok = pwait_warp(&sh.q_empty[buf], (fills[buf] & 1) ^ 1, &sh.abort);
        if (!ok) break;
        ++fills[buf];
        constexpr int CPR = D / 8, STEP = 32 / CPR;     // 16-byte pieces, rows per pass
        const int c = lane % CPR;
        int r = lane / CPR;
        int seq = s.gi, in_seq = first + r;
        if (s.kind == 0) {
          seq = s.gi * a.per + in_seq / a.gw;
          in_seq %= a.gw;
        }
        const uint32_t dst = q_buf + buf * C::TILE_BYTES + (c / 8) * C::HALF;
        const __nv_bfloat16* src = a.q + ((long long)seq * a.hq_w + s.h * a.gw + in_seq) * D + c * 8;
        for (; r < rows; r += STEP) {
          cp_async_16_full(dst + r * 128 + ((c % 8 ^ (r & 7)) << 4), src);
          in_seq += STEP;
          src += STEP * D;
          while (s.kind == 0 && in_seq >= a.gw) {       // on to the next sequence's rows
            in_seq -= a.gw;
            src += (long long)(a.hq_w - a.gw) * D;
          }
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.q_full[buf]));
      }
      if (!ok) break;
      if (!s.pair) turn ^= 1;
    }
  } else if (warp == 17) {
    // --------------------------------------------------------- K and V loads
    role_begin();
    int slot = 0, tile_count = 0;
    uint32_t phase = 0;
    int filled = 0;          // slots filled at least once
    bool ok = true;
    for (int at = 0; ok; ++at) {
      const Seg* sp = segment(at);
      ok = sp != nullptr;
      if (!ok || sp->kind < 0) break;
      const Seg s = *sp;
      done_with(at);
      int kt = 0, vt = 0;    // next K, V tile
      for (int x = 0; x < 2 * s.n; ++x) {
        const bool is_k = kt < s.n && s.k_at(kt) == x;
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
              if (runs)
                for (int i = 0; i < 32; ++i)
                  if (runs >> ((lane * 32 + i) / c.box_rows) & 1) bits |= 1u << i;
              sh.bad[tile_count % kMaskRing][lane] = bits;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.mask_full[tile_count % kMaskRing]));
            ++tile_count;
          }
          __syncwarp();
          if (lane < boxes * (D / 64)) {
            const int half = lane / boxes;
            tma_load_4d(dst + half * C::HALF + r * 128, map, half * 64,
                        (row0 + r) % c.page_size, s.h * c.zh, page, bar);
          }
        }
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
  } else if (warp == 16) {
    // ------------------------------------------------------------------ MMA
    // The whole warp walks, one lane issues.  Slots are used in ring order: a
    // running position serves K and V alike.
    role_begin();
    constexpr uint32_t kQk = mma_idesc(128, 128, false), kPv = mma_idesc(128, D, true);
    constexpr uint32_t kStep = C::TILE_BYTES >> 4;       // slots apart, in descriptor units
    const uint32_t on = elect_one();
    const uint64_t qd0 = smem_desc(q_buf, 16, 1024), kd0 = smem_desc(ring, 16, 1024);
    const uint64_t vd0 = smem_desc(ring, C::HALF, 1024);
    int slot = 0, turn = 0;
    uint32_t phase = 0, q_phase0 = 0, q_phase1 = 0, p_phase0 = 0, p_phase1 = 0;
    bool ok = true;
    auto next_slot = [&]() {
      if (++slot == C::SLOTS) {
        slot = 0;
        phase ^= 1;
      }
    };
    auto full = [&]() { return pwait_warp(&sh.full[slot], phase, &sh.abort); };
    auto qk = [&](int st, int buf) {
      const uint64_t qd = qd0 + buf * kStep, kd = kd0 + slot * kStep;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = (uint32_t)((k / 4) * C::HALF + (k % 4) * 32) >> 4;
        mma_ss(on, tmem + st * 128, qd + off, kd + off, kQk, k > 0);
      }
      mma_commit(on, smem_u32(&sh.s_full[st]));
    };
    auto pv = [&](int st, bool acc) {
      const uint64_t vd = vd0 + slot * kStep;
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        mma_ts(on, tmem + 256 + st * 128, tmem + st * 128 + k * 8, vd + (uint32_t)(k * 2048 >> 4),
               kPv, acc || k > 0);
    };
    auto release = [&]() { mma_commit(on, smem_u32(&sh.empty[slot])); };
    auto p_ready = [&](int st) {
      uint32_t& ph = st ? p_phase1 : p_phase0;
      const bool r = pwait_warp(&sh.p_ready[st], ph, &sh.abort);
      ph ^= 1;
      tc_fence_after();
      return r;
    };
    auto q_ready = [&](int buf) {
      uint32_t& ph = buf ? q_phase1 : q_phase0;
      const bool r = pwait_warp(&sh.q_full[buf], ph, &sh.abort);
      ph ^= 1;
      tc_fence_after();
      return r;
    };
    for (int at = 0; ok; ++at) {
      const Seg* sp = segment(at);
      ok = sp != nullptr;
      if (!ok) break;
      const int kind = sp->kind, n = sp->n, paired = sp->pair;
      if (kind < 0) break;
      done_with(at);
      if (paired) {
        // K0 for both, then per tile: V, next K, each used by A, then by B.
        if (!(ok = q_ready(0) && full())) break;
        qk(0, 0);
        if (!(ok = q_ready(1))) break;
        qk(1, 1);
        release();
        next_slot();
        for (int i = 0; i < n; ++i) {
          const bool more = i + 1 < n;
          const int vslot = slot;
          if (!(ok = p_ready(0) && full())) break;
          pv(0, i > 0);
          next_slot();
          if (more) {
            if (!(ok = full())) break;
            qk(0, 0);
          } else {
            mma_commit(on, smem_u32(&sh.o_final[0]));
            mma_commit(on, smem_u32(&sh.q_empty[0]));
          }
          if (!(ok = p_ready(1))) break;
          const int kslot = slot;
          slot = vslot;
          pv(1, i > 0);
          release();
          slot = kslot;
          if (more) {
            qk(1, 1);
            release();
            next_slot();
          } else {
            mma_commit(on, smem_u32(&sh.o_final[1]));
            mma_commit(on, smem_u32(&sh.q_empty[1]));
          }
        }
      } else {
        // Streams take the tiles in turn: K0, K1, then V0, K2, V1, K3, ...
        const int buf = turn;
        turn ^= 1;
        if (!(ok = q_ready(buf) && full())) break;
        qk(0, buf);
        release();
        next_slot();
        if (n > 1) {
          if (!(ok = full())) break;
          qk(1, buf);
          release();
          next_slot();
        }
        if (n <= 2) mma_commit(on, smem_u32(&sh.q_empty[buf]));
        for (int i = 0; i < n; ++i) {
          const int st = i & 1;
          if (!(ok = p_ready(st) && full())) break;
          pv(st, i > 1);
          release();
          next_slot();
          if (i + 2 < n) {
            if (!(ok = full())) break;
            qk(st, buf);
            release();
            next_slot();
            if (i + 3 == n) mma_commit(on, smem_u32(&sh.q_empty[buf]));
          } else {
            mma_commit(on, smem_u32(&sh.o_final[st]));
          }
        }
      }
    }
    if (!ok) {   // given up: the products in flight end before tensor memory is freed
      mma_commit(on, smem_u32(&sh.drain));
      mbar_wait(smem_u32(&sh.drain), 0, kWaitLimitCycles);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- softmax
    take_registers();
    const int st = warp >> 3, half = warp >> 2 & 1, row = (warp & 3) * 32 + lane;
    const int pair_id = 1 + st * 4 + (warp & 3);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // TMEM lane of the warp's first row
    const uint32_t tS = tmem + lanes + st * 128, tO = tmem + lanes + 256 + st * 128 + half * (D / 2);
    float* mine = &sh.exchange[st][half][row];
    const float* other = &sh.exchange[st][half ^ 1][row];
    const uint64_t scale2 = pack2(__float_as_uint(a.scale_log2), __float_as_uint(a.scale_log2));
    int ring0 = 0, tiles0 = 0;                 // ring position, paged tiles before the segment
    uint32_t s_phase = 0, o_phase = 0;
    bool ok = true;
    for (int at = 0; ok; ++at) {
      const Seg* sp = segment(at);
      if (!sp || sp->kind < 0) break;
      const Seg s = *sp;
      done_with(at);
      const int steps = s.steps(st);
      const int rt = s.rt + (s.pair ? st : 0);
      const int rows = min(kTile, a.rows[s.kind] - rt * kTile);
      const int sr = a.slot_rows[s.kind];
      const long long slot = (long long)s.slot * 2 + st;
      float2* ml = a.ws_ml[s.kind] + slot * sr;
      const bool paged = a.cache[s.kind].page_table != nullptr;
      if (steps == 0 && half == 0 && row < rows) ml[row] = make_float2(-INFINITY, 0.f);
      const bool live = (warp & 3) * 32 < rows;           // the warp has rows
      const int t_row = s.kind ? (rt * kTile + row) % a.w : 0;   // window row of this row
      float m = -INFINITY;
      uint64_t sum[2] = {0, 0};
      for (int step = 0; step < steps; ++step) {
        const int tl = s.tile(st, step), t = s.t0 + tl;
        const bool window = s.kind && t >= s.hist;
        // Columns [0, lim) of this thread's 64 count.
        const int lim = (window ? min(a.w, t_row + 1) - (t - s.hist) * kTile : s.len - t * kTile) -
                        half * 64;
        ok = pwait_warp(&sh.s_full[st], s_phase, &sh.abort);
        if (!ok) break;
        s_phase ^= 1;
        tc_fence_after();
        if (paged && !window) {
          ok = pwait_warp(&sh.mask_full[(tiles0 + tl) % kMaskRing],
                          ((tiles0 + tl) / kMaskRing) & 1, &sh.abort);
          if (!ok) break;
        }
        if (live) {
          uint32_t x0[32], x1[32], p[32];
          auto load = [&]() {
            tmem_ld32(tS + half * 64, x0);
            tmem_ld32(tS + half * 64 + 32, x1);
            tc_wait_ld();
            if (__any_sync(0xffffffffu, lim < 64)) {
              mask32(x0, lim);
              mask32(x1, lim - 32);
            }
            if (paged && !window) {
              const int k = (tiles0 + tl) % kMaskRing;
              const unsigned b0 = sh.bad[k][2 * half], b1 = sh.bad[k][2 * half + 1];
              if (b0 | b1) {
                mask_bits(x0, b0);
                mask_bits(x1, b1);
              }
            }
          };
          auto exps = [&](uint64_t (&to)[2]) {
            const float ms = m == -INFINITY ? 0.f : -m;
            const uint64_t mm = pack2(__float_as_uint(ms), __float_as_uint(ms));
            float top0 = -INFINITY, top1 = -INFINITY;
            exp32(x0, scale2, mm, to, top0, p);
            exp32(x1, scale2, mm, to, top1, p + 16);
            return fmaxf(top0, top1) * a.scale_log2;
          };
          load();
          // The reference maximum m moves only when a tile exceeds it by
          // more than a factor 2^8, so P is formed with the old one while
          // the tile's maximum is still being taken; where it does move (the
          // first tile, then rarely), S, not overwritten yet, is read again.
          bool again = true;
          float top;
          if (step == 0) {
            top = max32(x1, max32(x0, -INFINITY)) * a.scale_log2;
          } else {
            uint64_t to[2] = {sum[0], sum[1]};
            top = exps(to);
            // Also the point after which P may overwrite S: both threads of
            // a row have read it.
            again = pair_any(pair_id, m == -INFINITY ? top > m : top > m + kLazyRescale);
            if (!again) {
              sum[0] = to[0];
              sum[1] = to[1];
            }
          }
          if (again) {
            *mine = top;
            named_bar_sync(pair_id, 64);
            top = fmaxf(top, *other);
            const bool up = m == -INFINITY ? top > m : top > m + kLazyRescale;
            const float f = up ? ex2(m - top) : 1.f;
            if (up) m = top;
            const uint64_t f2 = pack2(__float_as_uint(f), __float_as_uint(f));
            sum[0] = fma2(sum[0], f2, 0);
            sum[1] = fma2(sum[1], f2, 0);
            if (step > 0) {
              // The product that wrote O was issued before the one that
              // signalled S: it is complete.
#pragma unroll
              for (int c = 0; c < D / 64; ++c) {
                uint32_t o[32];
                tmem_ld32(tO + c * 32, o);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st32(tO + c * 32, o);
              }
            }
            load();
            named_bar_sync(pair_id, 64);   // both have read S again
            exps(sum);
          }
          tmem_st32(tS + half * 32, p);
          tc_wait_st();
        }
        // V rows behind the end hold whatever the cache holds there, NaN
        // included: 0 * NaN must not reach O.
        const int valid = s.len - t * kTile;
        if (!window && valid < kTile && (!s.pair || st == 0)) {
          const int vat = ring0 + s.v_at(tl);
          ok = pwait_warp(&sh.full[vat % C::SLOTS], (vat / C::SLOTS) & 1, &sh.abort);
          if (!ok) break;
          const uint32_t v = ring + vat % C::SLOTS * C::TILE_BYTES;
          for (int i = valid * 8 + half * 128 + row; i < kTile * 8; i += 256)
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};\n" ::"r"(v + c * C::HALF +
                                                                              i * 16),
                           "r"(0)
                           : "memory");
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.p_ready[st]));
      }
      if (!ok) break;
      ring0 += 2 * s.n;
      if (paged) tiles0 += max(0, min(s.t0 + s.n, s.hist) - s.t0);
      if (steps == 0) continue;
      ok = pwait_warp(&sh.o_final[st], o_phase, &sh.abort);
      if (!ok) break;
      o_phase ^= 1;
      tc_fence_after();
      if (live) {
        // Pieces of four columns, rows side by side: full lines per store.
        float* out = a.ws_o[s.kind] + slot * sr * D + (long long)(half * (D / 8)) * sr * 4 + row * 4;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + c * 32, o);
          tc_wait_ld();
          if (row < rows) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4*>(out + (c * 8 + i / 4) * (sr * 4)) =
                  make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
        const uint64_t all = add2(sum[0], sum[1]);
        const float l = lo_of(all) + hi_of(all);
        if (half) *mine = l;
        named_bar_sync(pair_id, 64);
        if (!half && row < rows) ml[row] = make_float2(m, l + *other);
        named_bar_sync(pair_id, 64);   // read before the next segment writes
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) tmem_dealloc<512>(tmem);
}

// ---- combine: one thread per four columns of an output row

struct CombineArgs {
  PrefixKArgs k;
  __nv_bfloat16* o;
  float* lse;
  long long rows;      // b * h_q * w
};

constexpr int kCombineThreads = 256;

template <int D>
__global__ void __launch_bounds__(kCombineThreads)
    attn_prefix_combine_kernel(const __grid_constant__ CombineArgs c) {
  constexpr int ROWS = kCombineThreads / (D / 4);
  const PrefixKArgs& a = c.k;
  const int piece = threadIdx.x / ROWS;
  const long long row = (long long)blockIdx.x * ROWS + threadIdx.x % ROWS;
  griddep_wait();
  griddep_launch_dependents();
  if (row >= c.rows) return;
  const int seq = (int)(row / a.hq_w), in_seq = (int)(row % a.hq_w);
  const int h = in_seq / a.gw, r = in_seq % a.gw;
  const Cut cut(a.plan[0], a.grid);
  // Partials of the row in its prefix item and in its own: CTAs first ..
  // first + ctas - 1, one stream of a pair's slot or both of a single's.
  int ctas[2], twice[2];
  long long at[2];
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const int gi = kind ? seq : seq / a.per;
    const int rr = kind ? r : seq % a.per * a.gw + r;
    const int rt = rr / kTile, pairs = a.row_tiles[kind] >> 1, set = rt >> 1;
    const bool pair = set < pairs;
    const int tiles = tiles_of(a, kind, length_of(a, kind, gi));
    ctas[kind] = 0;
    twice[kind] = pair ? 0 : 1;
    if (tiles > 0) {
      const int start = a.plan[1 + kind * a.count[0] + gi] +
                        (h * a.row_tiles[kind] + set * 2) * tiles;
      const int first = cut.of(start);
      ctas[kind] = cut.of(start + (tiles - 1) * (pair ? 2 : 1)) - first + 1;
      const int item = (gi * a.hkv + h) * ((a.row_tiles[kind] + 1) >> 1) + set;
      at[kind] = (long long)(first + item) * 2 + (pair ? rt & 1 : 0);
    }
  }
  float top = -INFINITY;
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const int sr = a.slot_rows[kind], in_tile = (kind ? r : seq % a.per * a.gw + r) % kTile;
    const int n = ctas[kind] << twice[kind], stride = 2 - twice[kind];
#pragma unroll 4
    for (int i = 0; i < n; ++i)
      top = fmaxf(top, a.ws_ml[kind][(at[kind] + i * stride) * sr + in_tile].x);
  }
  const float m = top == -INFINITY ? 0.f : top;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const int sr = a.slot_rows[kind], in_tile = (kind ? r : seq % a.per * a.gw + r) % kTile;
    const int n = ctas[kind] << twice[kind], stride = 2 - twice[kind];
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const long long base = (at[kind] + i * stride) * sr;
      const float2 ml = a.ws_ml[kind][base + in_tile];
      const float4 v = *reinterpret_cast<const float4*>(a.ws_o[kind] + base * D +
                                                        ((long long)piece * sr + in_tile) * 4);
      const float wt = ex2(ml.x - m);
      if (wt > 0.f) {   // otherwise nothing was seen there (O may be unwritten)
        l = fmaf(wt, ml.y, l);
        acc.x = fmaf(wt, v.x, acc.x);
        acc.y = fmaf(wt, v.y, acc.y);
        acc.z = fmaf(wt, v.z, acc.z);
        acc.w = fmaf(wt, v.w, acc.w);
      }
    }
  }
  const float inv = top == -INFINITY ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(c.o + row * D + piece * 4) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (piece == 0) c.lse[row] = top == -INFINITY ? -INFINITY : (m + log2f(l)) * kLn2;
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
  cudaError_t e = ensure_smem_attr(kern, kSmem<D>, done);
  if (e != cudaSuccess) return e;
  static std::atomic<int> split_ok{0};
  if ((e = check_register_split<Split>(kern, split_ok)) != cudaSuccess) return e;
  e = launch_pdl(kern, dim3((unsigned)k.grid), dim3(kThreads), kSmem<D>, st, k, maps);
  if (e != cudaSuccess) return e;
  note_launches(1);
  constexpr int kRows = kCombineThreads / (D / 4);
  CombineArgs c{};
  c.k = k;
  c.o = p.o;
  c.lse = p.lse;
  c.rows = (long long)p.b * p.hq * p.w;
  e = launch_pdl(attn_prefix_combine_kernel<D>,
                 dim3((unsigned)((c.rows + kRows - 1) / kRows)), dim3(kCombineThreads), 0, st, c);
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
