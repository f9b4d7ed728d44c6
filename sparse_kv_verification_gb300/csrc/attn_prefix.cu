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
// One persistent CTA per SM; lengths are on the device, so every CTA works
// out its share itself (Walk).  Prefixes are split: each row tile pair's
// tiles into np equal segments, the single's into ns (fewer, as its tiles
// cost less), one segment to a CTA, np and ns from the M (cost of the tiles of
// a segment) whose longest CTA is the shortest.  All pairs walk
// the same K/V tiles at the same time: a prefix of 32768 positions is as
// large as L2, and with the row tiles one after another it came from HBM once
// per pair of them (512 rows: 64 instead of 44 us for the loads alone).  The
// own items lie on a line that the remaining CTAs share in equal ranges, cut
// into segments no longer than a range, so that at most two CTAs share one.
// Where a split leaves CTAs idle too long, the prefixes go on the line too.
// Partial results (O unnormalised, m, l) go to the workspace, each segment
// (on the line: each of two parts) has its place, and
// attn_prefix_combine_kernel adds each row's partials in a fixed order.
//
// Roles of the 16 warps: 0 issues tcgen05.mma, 1 and 7 the TMA loads of K and
// V, 2 walks the CTA's share and publishes its segments, 3 (of CTA 0) writes
// the plan for the combine kernel, 4-6 copy Q rows, 8-11 and 12-15 are the
// softmax of stream A and B, one thread per row.  S = Q K^T and O += P V
// accumulate in tensor memory (512 columns: per stream an S of 128 positions
// and an O); P replaces S in place as bf16, half by half, and is read from
// there as the A operand, so only Q, K and V live in shared memory.  While one
// stream's softmax works, the tensor cores work for the other.
#include <algorithm>
#include <climits>

#include "device_common.cuh"
#include "dustin.h"
#include "internal.h"
#include "quotient.h"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace dustin {

namespace {

__device__ unsigned int g_prefix_dev_flags;

constexpr int kTile = 128;        // positions of a K/V tile, rows of a row tile
constexpr int kHalf = 64;         // positions whose P is handed over at a time
constexpr int kSoftmaxWarps = 4;  // per stream
constexpr int kMmaWarp = 0, kLoadWarp = 1, kWalkWarp = 2, kTableWarp = 3, kQWarp = 4, kQWarps = 3,
              kLoadWarp2 = 7, kSoftmaxWarp = 8;
constexpr int kThreads = 16 * 32;
// Registers: a softmax thread holds 64 scores and their weights; the other
// two warpgroups give up what they need beyond the launch's 128.
struct Split {
  static constexpr int NT = kThreads, NPW = 8, NCW = 2 * kSoftmaxWarps;
  static constexpr int PRODUCER_REGS = 112, CONSUMER_REGS = 144;
};
// Weights of one half tile's row may add up to this.
constexpr float kMostWeight = 256.f;
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
  int pages_per_seq, num_pages;
  int runs;            // runs per page
  int zh, zb;          // 0 where that stride is 0: the coordinate stays 0
};

struct PrefixKArgs {
  const __nv_bfloat16* q;
  const int* prefix_len;
  const int* own_len;
  float* ws_o[2];      // partial O: prefix slots, own slots
  float2* ws_ml[2];
  int* plan;           // see kPlanInts
  PrefixCache cache[3];
  int n[2];            // prefix, own positions at most
  int count[2];        // groups, sequences
  int row_tiles[2];    // of a prefix, own item family
  int rows[2];         // rows of one (group or sequence, kv head)
  int slot_rows[2];    // rows per stream of a partial's place
  int streams[2];      // streams per place (2 where the family has pairs)
  int log_box[2];      // of the family's tiles, the window's included
  int per, gw, hq_w, hkv, w, win_tiles, grid;
  // Prefixes of one length: CTAs that have one segment of them each, segments
  // of a pair and of the single.  0: decided on the device, where the lengths
  // are.
  int split, np, ns;
  int range;           // with split > 0 and own parts of one length: the line's
  float inv_grid, scale_log2;
  float inv_per, inv_gw, inv_hq_w;   // for quotient()
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
  int slot;            // place of its partials
  int whole;           // on the line, not shared: the place behind it stays empty
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

// Shared-memory layout of a V tile: boxes of 2^log_box rows behind one
// another, each with its 64-column halves behind one another.  (A K tile has
// its halves of all 128 rows behind one another: rows that are a product's N
// lie at one stride.)
template <int D>
__device__ __forceinline__ uint32_t v_row(int row, int log_box) {
  return (uint32_t)((row >> log_box) << (log_box + (D == 128 ? 8 : 7))) +
         (uint32_t)((row & ((1 << log_box) - 1)) << 7);
}

struct Control {
  float2 exchange[2][kTile];       // m, l of a single's streams
  unsigned long long full[10], empty[10];
  unsigned long long q_full[2], q_empty[2], s_full[2], p_ready[2][2], half_done[2], o_final[2];
  unsigned long long seg_full[kSegRing], seg_empty[kSegRing], mask_full[kMaskRing], meet, drain;
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

// try_wait that may keep the thread suspended for up to 100 us.
__device__ __forceinline__ bool try_wait_long(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(100000u)
      : "memory");
  return ok != 0;
}
// Waits with the library's limit; gives up when another role has.  Suspended,
// not polling: waiting warps otherwise take the issue slots of those at work.
__device__ __forceinline__ bool pwait(unsigned long long* bar, uint32_t parity, int* abort) {
  const uint32_t b = smem_u32(bar);
  if (mbar_try_wait(b, parity)) return true;
  const long long t0 = clock64();
  while (!try_wait_long(b, parity)) {
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
// Of the quotients below (quotient.h), those of the whole line by some CTAs have
// no bound but the line's length (below 2^28), where the CTAs are few: on devices
// of a few SMs, or where a split leaves few.  The others are counts of tiles,
// heads, sequences or CTAs, which the host's limits keep below 2^22.

// Work is counted in eighths of a pair's K/V tile.  A tile for one row tile
// alone costs more than half of that (its K and V come for it alone, and its
// two streams wait for one another's tensor core time less evenly), and a
// segment as much as two tiles beside its own: its Q, its start and end, its
// partials and their part in the combination.  Measured: with 8 for a segment
// 32 sequences of four ragged prefixes take 89 instead of 75 us, a 7B-shaped
// step 28 instead of 25, two short sequences 13.7 instead of 10.3; with 24, 64
// sequences with short own parts take 70 instead of 66.
constexpr int kPairCost = 8, kSingleCost = 5, kSegmentCost = 18;
// One K/V tile for rt row tiles.
__host__ __device__ constexpr int tile_cost(int rt) { return (rt >> 1) * kPairCost + (rt & 1) * kSingleCost; }
// A range holds a segment of two tiles of a single (a few own positions and the
// window) or one of a pair at least: with one tile, two short sequences take
// 11.7 instead of 9.6 us.
constexpr int kMinRange = kSegmentCost + 2 * kSingleCost;
static_assert(kMinRange >= kSegmentCost + kPairCost, "a segment fits a range");

// The line cut into n ranges of at least kMinRange: range c starts at
// ceil(c * total / n), which is c * (total / n) + ceil(c * (total % n) / n),
// all in 32 bits.
struct Cut {
  int n, total, q, r;
  float inv;
  __device__ __forceinline__ Cut(int line, int ctas) {
    total = line;
    n = max(1, min(ctas, total / kMinRange));
    inv = reciprocal(n);
    q = quotient_wide(total, n, inv);
    r = total - q * n;
  }
  __device__ __forceinline__ int start(int c) const {
    return c >= n ? total : c * q + quotient(c * r + n - 1, n, inv);
  }
};

// Whether an equal share on the line, two segments to a CTA, ends before a
// split that takes `longest`, for items whose row tiles all share their K/V
// tiles anyway.
__host__ __device__ constexpr bool on_line_is_shorter(long long longest, long long share) {
  return longest > share + share / 16 + 2 * kSegmentCost;
}

// A segment's tiles on the line: n of them, w apart, then its fixed cost.
struct Span {
  int pos, n, w;
  __device__ __forceinline__ int length() const { return n * w + kSegmentCost; }
  // The first tile at or behind a cut at b.  A cut that would leave a piece
  // shorter than `snap` moves to the segment's end.
  __device__ __forceinline__ int tile(int b, int snap) const {
    const int x = b - pos, len = length();
    if (x <= 0) return 0;
    if (x >= len) return n;
    if (x < snap && x <= len - x) return 0;
    if (len - x < snap) return n;
    return min(n, quotient_up(x, w));
  }
};

// Items of one family on the line: per (group or sequence, kv head) chunks of
// `chunk` tiles, each with one segment per set (pairs, then the single).
struct Family {
  int rt, pairs, sets, tile, chunk;
  float inv;
  __device__ __forceinline__ void set(const PrefixKArgs& a, int kind, int range) {
    rt = a.row_tiles[kind];
    pairs = rt >> 1;
    sets = (rt + 1) >> 1;
    tile = tile_cost(rt);
    // The most tiles whose segment fits a range.
    const int room = range - kSegmentCost;
    chunk = max(1, pairs ? room / kPairCost : room / kSingleCost);
    inv = reciprocal(chunk);
  }
  __device__ __forceinline__ int count(int tiles) const {
    return quotient(tiles + chunk - 1, chunk, inv);
  }
  // Length on the line of a chunk of m tiles; of all tiles of one kv head.
  __device__ __forceinline__ int chunk_length(int m) const { return m * tile + sets * kSegmentCost; }
  __device__ __forceinline__ int length(int tiles) const {
    return tiles * tile + count(tiles) * sets * kSegmentCost;
  }
  // Set y of a chunk of m tiles at pos.
  __device__ __forceinline__ Span segment(int m, int y, int pos) const {
    return {pos + y * (m * kPairCost + kSegmentCost), m, y < pairs ? kPairCost : kSingleCost};
  }
};

// Plan header: 1 where the prefixes are split; then for every group and
// sequence {first place, segments}: np | ns << 16 where split, else chunks.
constexpr int kPlanInts = 4;

// Walks the segments of this CTA.
struct Walk {
  const PrefixKArgs& a;
  Family fam;
  int snap, b0, b1, range;
  int m;                                // device search: the most a segment's tiles cost
  int kind, gi, h, c, y;
  int pos, place, len, tiles, chunks;   // pos, place: of chunk c and its first segment
  bool one;                             // a split CTA: its segment is in `only`
  Seg only;

  // Over one family: tiles (x) and, with a chunk set, chunks, else members
  // that have any (y).  t: of the first 32 members, one per lane.
  __device__ __forceinline__ int2 sums(int k, int t, const Family* f) const {
    const int lane = threadIdx.x & 31;
    int x = 0, y = 0;
    for (int i = lane; i < a.count[k]; i += 32) {
      if (i != lane) t = tiles_at(k, i);
      x += t;
      y += f ? f->count(t) : t > 0;
    }
#pragma unroll 1
    for (int d = 16; d > 0; d >>= 1) {
      x += __shfl_xor_sync(0xffffffffu, x, d);
      y += __shfl_xor_sync(0xffffffffu, y, d);
    }
    return make_int2(x, y);
  }
  __device__ __forceinline__ int tiles_at(int k, int i) const {
    return tiles_of(a, k, length_of(a, k, i));
  }

  // M by search: CTAs the prefixes take, 0 where they go on the line.  One
  // warp; t0: tiles of the first 32 groups.
  __device__ __forceinline__ int search(int t0, int wp, int wo) {
    const int lane = threadIdx.x & 31;
    const int rt = a.row_tiles[0], pairs = rt >> 1, single = rt & 1;
    if (wp == 0 || a.count[0] * a.hkv * ((rt + 1) >> 1) > a.grid) return 0;
    // Candidates from the even share on, lane 0 first.
    const int share = quotient_wide(wp + wo + a.grid - 1, a.grid, a.inv_grid);
    const int least = max(16, share);
    const int x = least + least / 24 * lane + least % 24 * lane / 24;   // by 24ths
    const float inv = reciprocal(x);
    int ctas = 0;
    for (int g = 0; g < a.count[0]; ++g) {
      const int t = g < 32 ? __shfl_sync(0xffffffffu, t0, g) : tiles_at(0, g);
      ctas += pairs * quotient_up(t * kPairCost, x, inv) + single * quotient_up(t * kSingleCost, x, inv);
    }
    ctas *= a.hkv;
    const int own = a.grid - ctas;       // CTAs left
    const bool fits = wo ? own > 0 : own >= 0;
    const unsigned longest =
        fits ? (unsigned)max(x + kSegmentCost, wo ? quotient_wide(wo + own - 1, own) : 0) : ~0u;
    const unsigned least_of = __reduce_min_sync(0xffffffffu, longest);
    if (least_of == ~0u) return 0;
    const int src = __ffs((int)__ballot_sync(0xffffffffu, longest == least_of)) - 1;
    m = __shfl_sync(0xffffffffu, x, src);
    if (rt <= 2 && on_line_is_shorter(least_of, share)) return 0;
    return __shfl_sync(0xffffffffu, ctas, src);
  }
  // The one segment of a split CTA, the x-th of group gi.  Of a kv head: for
  // each of the np parts all pairs, then the single's.
  __device__ __forceinline__ void direct(int x, int np, int ns) {
    const int rt = a.row_tiles[0], pairs = rt >> 1, per = pairs * np + ns;
    len = length_of(a, 0, gi);
    tiles = (len + kTile - 1) / kTile;
    h = quotient(x, per);
    const int z = x - h * per;
    only.kind = 0;
    only.gi = gi;
    only.h = h;
    only.pair = z < pairs * np;
    const int part = only.pair ? quotient(z, pairs) : z - pairs * np;
    const int parts = only.pair ? np : ns;
    const float inv = reciprocal(parts);
    only.rt = only.pair ? 2 * (z - part * pairs) : rt - 1;
    only.t0 = quotient(part * tiles, parts, inv);
    only.n = quotient((part + 1) * tiles, parts, inv) - only.t0;
    only.len = len;
    only.hist = tiles;
    only.slot = blockIdx.x;
    only.whole = 0;
    one = true;
    pos = b1 = 0;
  }
  // On the line: from the sequence (or group) at pos to the segment at b0.
  __device__ __forceinline__ void seek() {
    if (b0 >= b1) {
      pos = b1;   // nothing here
      return;
    }
    load();
    const int per = fam.length(tiles);
    h = quotient(b0 - pos, per);
    pos += h * per;
    const int full = fam.chunk_length(fam.chunk);
    c = min(quotient(b0 - pos, full), chunks - 1);
    pos += c * full;
    place += (h * chunks + c) * fam.sets * 2;
  }

  // One warp.  With `write` (one warp of the grid) it leaves the plan for the
  // combine kernel instead of looking for this CTA's share.
  __device__ Walk(const PrefixKArgs& args, bool write) : a(args) {
    const int lane = threadIdx.x & 31, cta = blockIdx.x;
    int2* table = reinterpret_cast<int2*>(a.plan + kPlanInts);
    kind = gi = pos = place = h = c = y = 0;
    one = false;
    if (a.split > 0) {
      // Prefixes of one length, split by the host.
      const int per_group = a.hkv * ((a.row_tiles[0] >> 1) * a.np + a.ns);
      if (write) {
        if (lane == 0) a.plan[0] = 1;
        for (int g = lane; g < a.count[0]; g += 32)
          table[g] = make_int2(g * per_group, a.np | a.ns << 16);
      } else if (cta < a.split) {
        gi = quotient(cta, per_group);
        direct(cta - gi * per_group, a.np, a.ns);
        return;
      }
      if (a.own_len == nullptr) {
        // Own parts of one length too: all in closed form.
        kind = 1;
        range = a.range;
        load();
        const int per = fam.length(tiles) * a.hkv, places = chunks * fam.sets * a.hkv * 2;
        if (write) {
          for (int i = lane; i < a.count[1]; i += 32)
            table[a.count[0] + i] = make_int2(i * places, chunks);
          return;
        }
        const Cut cut(per * a.count[1], max(a.grid - a.split, 1));
        snap = cut.q >> 4;
        b0 = cut.start(cta - a.split);
        b1 = cut.start(cta - a.split + 1);
        gi = per ? quotient(b0, per) : 0;
        pos = gi * per;
        place = gi * places;
        seek();
        return;
      }
    }
    // This lane's group and sequence (the first 32).
    const int t0 = lane < a.count[0] && a.split == 0 ? tiles_at(0, lane) : 0;
    const int t1 = lane < a.count[1] ? tiles_at(1, lane) : 0;
    const int2 s1 = sums(1, t1, nullptr);
    int on_line = a.hkv * (s1.x * tile_cost(a.row_tiles[1]) +
                           s1.y * ((a.row_tiles[1] + 1) >> 1) * kSegmentCost);
    int split = a.split;
    if (split == 0) {
      const int wp = sums(0, t0, nullptr).x * a.hkv * tile_cost(a.row_tiles[0]);
      split = search(t0, wp, on_line);
      if (!split) on_line += wp;
      if (write && lane == 0) a.plan[0] = split ? 1 : 0;
    }
    // A lower bound of the ranges' length, the line's length.
    const int ctas = max(a.grid - split, 1);
    range = max(kMinRange, quotient_wide(on_line, ctas));
    int total = 0;
#pragma unroll 1
    for (int k = split ? 1 : 0; k < 2; ++k) {
      fam.set(a, k, range);
      const int2 x = sums(k, k ? t1 : t0, &fam);
      total += a.hkv * (x.x * fam.tile + x.y * fam.sets * kSegmentCost);
    }
    const Cut cut(total, ctas);
    snap = cut.q >> 4;
    const bool in_split = cta < split && !write;
    b0 = in_split ? 0 : cut.start(max(cta - split, 0));
    b1 = in_split ? 0 : cut.start(max(cta - split, 0) + 1);
    int base = 0;
#pragma unroll 1
    for (int k = a.split > 0 ? 1 : 0; k < 2; ++k) {
      const bool is_split = k == 0 && split;
      int places = 0;
      fam.set(a, k, range);
      for (int i0 = 0; i0 < a.count[k]; i0 += 32) {
        const int i = i0 + lane;
        const int t = i0 ? (i < a.count[k] ? tiles_at(k, i) : 0) : (k ? t1 : t0);
        // Its length on the line (split: nothing), its places, its segments.
        int length = 0, mine = 0, segs = 0;
        if (is_split) {
          const int pairs = a.row_tiles[0] >> 1;
          const int np = pairs ? quotient_up(t * kPairCost, m) : 0;
          const int ns = a.row_tiles[0] & 1 ? quotient_up(t * kSingleCost, m) : 0;
          mine = (pairs * np + ns) * a.hkv;
          segs = np | ns << 16;
        } else {
          segs = fam.count(t);
          length = fam.length(t) * a.hkv;
          mine = segs * fam.sets * a.hkv * 2;
        }
        int at = length, pl = mine;
#pragma unroll 1
        for (int d = 1; d < 32; d <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, at, d), w = __shfl_up_sync(0xffffffffu, pl, d);
          if (lane >= d) {
            at += v;
            pl += w;
          }
        }
        const int all = __shfl_sync(0xffffffffu, at, 31), all_places = __shfl_sync(0xffffffffu, pl, 31);
        at += base - length;
        pl += places - mine;
        if (write) {
          if (i < a.count[k]) table[k * a.count[0] + i] = make_int2(pl, segs);
        } else {
          const bool hit = is_split ? in_split && pl <= cta && cta < pl + mine
                                    : !in_split && at <= b0 && b0 < at + length;
          const unsigned here = __ballot_sync(0xffffffffu, hit);
          if (here) {
            const int src = __ffs((int)here) - 1;
            kind = k;
            gi = i0 + src;
            pos = __shfl_sync(0xffffffffu, at, src);
            place = __shfl_sync(0xffffffffu, pl, src);
            const int x = __shfl_sync(0xffffffffu, segs, src);
            if (is_split)
              direct(cta - place, x & 0xffff, x >> 16);
            else
              seek();
            return;
          }
        }
        base += all;
        places += all_places;
      }
    }
    pos = b1;   // nothing here
  }
  __device__ __forceinline__ void load() {
    fam.set(a, kind, range);
    len = length_of(a, kind, gi);
    tiles = tiles_of(a, kind, len);
    chunks = fam.count(tiles);
  }
  __device__ bool next(Seg& s) {
    if (one) {
      s = only;
      one = false;
      return s.n > 0;
    }
    while (pos < b1) {
      if (tiles == 0 || h == a.hkv) {
        h = 0;
        if (++gi == a.count[kind]) {
          gi = 0;
          place = 0;
          ++kind;      // pos < b1 <= total: there is work left in family 1
        }
        load();
        continue;
      }
      const int m = min(fam.chunk, tiles - c * fam.chunk);
      const Span sp = fam.segment(m, y, pos);
      const int lo = sp.tile(b0, snap), hi = sp.tile(b1, snap);
      s.kind = kind;
      s.gi = gi;
      s.h = h;
      s.pair = y < fam.pairs;
      s.rt = 2 * y;
      s.slot = place + 2 * y + (lo > 0);
      s.whole = hi - lo == sp.n;
      s.t0 = c * fam.chunk + lo;
      s.n = hi - lo;
      s.len = len;
      s.hist = (len + kTile - 1) / kTile;
      const bool found = lo < hi;
      const bool past = sp.pos >= b1;
      if (++y == fam.sets) {
        y = 0;
        place += fam.sets * 2;
        pos += fam.chunk_length(m);
        if (++c == chunks) {
          c = 0;
          ++h;
        }
      }
      if (found) return true;
      if (past) break;
    }
    pos = b1;
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
// The largest of 32 scores and top.
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
// p = 2^(x * scale - m) as 16 bf16 pairs, the fp32 values added to sum.
__device__ __forceinline__ void exp32(const uint32_t (&x)[32], uint64_t scale, uint64_t minus_m,
                                      uint64_t (&sum)[2], uint32_t* p) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint64_t y = fma2(pack2(x[2 * i], x[2 * i + 1]), scale, minus_m);
    const float e0 = ex2(lo_of(y)), e1 = ex2(hi_of(y));
    sum[i & 1] = add2(sum[i & 1], pack2(__float_as_uint(e0), __float_as_uint(e1)));
    // P in bf16, as the tensor cores take it (relative rounding 2^-8 per
    // weight); the row sum keeps the fp32 values.
    p[i] = pack_bf16(e0, e1);
  }
}
// Columns whose bits are set do not count.
__device__ __forceinline__ void mask_bits(uint32_t (&x)[32], unsigned dead) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (dead >> i & 1) x[i] = 0xff800000u;   // -inf
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
      mbar_init(smem_u32(&sh.full[i]), 2);   // both load warps
      mbar_init(smem_u32(&sh.empty[i]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sh.q_full[s]), kQWarps);
      mbar_init(smem_u32(&sh.q_empty[s]), 1);
      mbar_init(smem_u32(&sh.s_full[s]), 1);
      mbar_init(smem_u32(&sh.half_done[s]), 1);
      for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sh.p_ready[s][i]), kSoftmaxWarps);
      mbar_init(smem_u32(&sh.o_final[s]), 1);
    }
    for (int i = 0; i < kMaskRing; ++i) mbar_init(smem_u32(&sh.mask_full[i]), 1);
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(smem_u32(&sh.seg_full[i]), 1);
      mbar_init(smem_u32(&sh.seg_empty[i]), 2 * kSoftmaxWarps + 3 + kQWarps);
    }
    mbar_init(smem_u32(&sh.meet), 2 * kSoftmaxWarps);
    mbar_init(smem_u32(&sh.drain), 1);
    mbar_fence_init();
    sh.abort = 0;
  }
  if (warp == kMmaWarp) tmem_alloc<512>(smem_u32(&sh.tmem));
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

  if (warp < kSoftmaxWarp) give_registers();   // one instruction for whole warpgroups
  if (warp == kWalkWarp) {
    // --------------------------------------------------------------- walker
    role_begin();
    Walk walk(a, false);
    Seg s{};
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
  } else if (warp == kTableWarp) {
    role_begin();
    if (blockIdx.x == 0) Walk(a, true);
  } else if (warp >= kQWarp && warp < kQWarp + kQWarps) {
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
        constexpr int CPR = D / 8, STEP = 32 * kQWarps / CPR;   // 16-byte pieces, rows per pass
        const int piece = tid - kQWarp * 32, c = piece % CPR;
        const uint32_t dst = q_buf + buf * C::TILE_BYTES + (c / 8) * C::HALF;
        const __nv_bfloat16* src = a.q + (long long)s.h * a.gw * D + c * 8;
        for (int r = piece / CPR; r < rows; r += STEP) {
          int seq = s.gi, in_seq = first + r;
          if (s.kind == 0) {
            const int rr = in_seq;
            int q = (int)((float)rr * a.inv_gw);        // at most one off
            q -= q * a.gw > rr;
            q += (q + 1) * a.gw <= rr;
            seq = s.gi * a.per + q;
            in_seq = rr - q * a.gw;
          }
          cp_async_16_full(dst + r * 128 + ((c % 8 ^ (r & 7)) << 4),
                           src + ((long long)seq * a.hq_w + in_seq) * D);
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
  } else if (warp == kLoadWarp || warp == kLoadWarp2) {
    // --------------------------------------------------------- K and V loads
    // Two warps, each with half of a tile's boxes: a warp's lanes issue their
    // boxes one after another (pages of 16 make 24 of them a tile: with one warp
    // own parts on such pages were read at 5.0 TB/s, with two at 6.0).  Both
    // arrive on every slot, the second one also where it has no box of the tile
    // (tiles of one box: no half of V, at d 64 none of K either): a warp that
    // fell a lap of the ring behind would wait for a phase already gone.
    role_begin();
    const bool second = warp == kLoadWarp2;
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
      const PrefixCache& cache = a.cache[s.kind];
      const int log_box = a.log_box[s.kind], boxes = kTile >> log_box;
      // Lane l loads run l % boxes of a tile, half l / boxes.  Its page: of
      // the next K tile, and of the up to two tiles whose V is still to come.
      const int run = lane & (boxes - 1), half = lane >> (7 - log_box);
      auto page_of = [&](int t) -> int {
        const int j = t * kTile + (run << log_box);
        if (!cache.page_table || j >= s.len) return cache.num_pages;   // loads as zeros
        const int x = j >> log_box;
        return __ldg(cache.page_table + (long long)s.gi * cache.pages_per_seq +
                     (cache.runs == 1 ? x : x / cache.runs));
      };
      int page_k = page_of(s.t0), page_v0 = 0, page_v1 = 0, pending = 0;
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
        int row = row0 + (run << log_box), outer = s.gi * c.zb;
        if (c.page_table) {
          int page = is_k ? page_k : page_v0;
          const bool in = row < s.len, bad = in && (page < 0 || page >= c.num_pages);
          if (is_k && !second) {
            // Positions on pages outside the pool, for the softmax.
            const unsigned all = __ballot_sync(0xffffffffu, bad && half == 0);
            if (lane < 4) {
              unsigned bits = 0;
              if (all)
                for (int i = 0; i < 32; ++i)
                  if (all >> ((lane * 32 + i) >> log_box) & 1) bits |= 1u << i;
              sh.bad[tile_count % kMaskRing][lane] = bits;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.mask_full[tile_count % kMaskRing]));
            ++tile_count;
            if (bad) raise_flag(DUSTIN_DEVFLAG_PAGE_RANGE);
          }
          // Past the map's extent: zeros.
          outer = in && !bad ? page * c.zb : c.num_pages;
          const int r = row >> log_box;
          row = c.runs == 1 ? 0 : (r - r / c.runs * c.runs) << log_box;
        }
        if (is_k) {
          if (pending)
            page_v1 = page_k;
          else
            page_v0 = page_k;
          ++pending;
          if (kt < s.n) page_k = page_of(s.t0 + kt);
        } else {
          page_v0 = page_v1;
          --pending;
        }
        if (lane == 0) {
          if (second)
            mbar_arrive(bar);
          else
            mbar_arrive_expect_tx(bar, C::TILE_BYTES);
        }
        __syncwarp();
        if (is_k) {
          if (half < D / 64 && (D == 128 ? half : run & 1) == second)
            tma_load_5d(dst + half * C::HALF + (run << (log_box + 7)), map, 0, row, half,
                        s.h * c.zh, outer, bar);
        } else if (half == 0 && (run & 1) == second) {
          tma_load_5d(dst + v_row<D>(run << log_box, log_box), map, 0, row, 0, s.h * c.zh, outer,
                      bar);
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
        if (!mbar_wait(smem_u32(&sh.full[slot]), phase, kWaitLimitCycles)) break;
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMA
    // The whole warp walks, one lane issues.  Slots are used in ring order: a
    // running position serves K and V alike.
    role_begin();
    constexpr uint32_t kQk = mma_idesc(128, kTile, false), kPv = mma_idesc(128, D, true);
    constexpr uint32_t kStep = C::TILE_BYTES >> 4;       // slots apart, in descriptor units
    const uint32_t on = elect_one();
    const uint64_t qd0 = smem_desc(q_buf, 16, 1024), kd0 = smem_desc(ring, 16, 1024);
    int slot = 0, turn = 0;
    uint32_t phase = 0, q_phase0 = 0, q_phase1 = 0, p_phase = 0;   // p_phase: a bit per stream
    bool ok = true;
    auto next_slot = [&]() {
      if (++slot == C::SLOTS) {
        slot = 0;
        phase ^= 1;
      }
    };
    auto full = [&]() { return pwait_warp(&sh.full[slot], phase, &sh.abort); };
    auto qk = [&](int st, int buf, int kslot) {
      const uint64_t qd = qd0 + buf * kStep, kd = kd0 + kslot * kStep;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = (uint32_t)((k / 4) * C::HALF + (k % 4) * 32) >> 4;
        mma_ss(on, tmem + st * 128, qd + off, kd + off, kQk, k > 0);
      }
      mma_commit(on, smem_u32(&sh.s_full[st]));
    };
    uint64_t vd0 = 0;                                    // by the segment's boxes
    int log_box = 7;
    auto pv = [&](int st, int x, int vslot, bool acc) {
      const uint64_t vd = vd0 + vslot * kStep;
#pragma unroll
      for (int k = 0; k < kHalf / 16; ++k)
        mma_ts(on, tmem + 256 + st * 128, tmem + st * 128 + x * (kHalf / 2) + k * 8,
               vd + (v_row<D>(x * kHalf + k * 16, log_box) >> 4), kPv, acc || k > 0);
    };
    auto release = [&](int at) { mma_commit(on, smem_u32(&sh.empty[at])); };
    // Both halves of P come once per tile: one phase for both.
    auto p_ready = [&](int st, int x) {
      const bool r = pwait_warp(&sh.p_ready[st][x], p_phase >> st & 1, &sh.abort);
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
      log_box = a.log_box[kind];
      vd0 = smem_desc(ring, 128u << log_box, 1024);
      if (paired) {
        // K0 for both, then per tile, A then B, V half by half and the next K.
        if (!(ok = q_ready(0) && full())) break;
        qk(0, 0, slot);
        if (!(ok = q_ready(1))) break;
        qk(1, 1, slot);
        release(slot);
        next_slot();
        for (int i = 0; ok && i < n; ++i) {
          const bool more = i + 1 < n;
          const int vslot = slot;
          int kslot = 0;
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            if (!(ok = ok && p_ready(st, 0))) break;
            if (st == 0) {
              if (!(ok = full())) break;
              next_slot();
            }
            pv(st, 0, vslot, i > 0);
            mma_commit(on, smem_u32(&sh.half_done[st]));
            if (!(ok = p_ready(st, 1))) break;
            pv(st, 1, vslot, true);
            if (st == 1) release(vslot);
            if (more) {
              if (st == 0) {
                if (!(ok = full())) break;
                kslot = slot;
                next_slot();
              }
              qk(st, st, kslot);
              if (st == 1) release(kslot);
            } else {
              mma_commit(on, smem_u32(&sh.o_final[st]));
              mma_commit(on, smem_u32(&sh.q_empty[st]));
            }
          }
          p_phase ^= 3;
        }
      } else {
        // Streams take the tiles in turn: K0, K1, then V0, K2, V1, K3, ...
        const int buf = turn;
        turn ^= 1;
        if (!(ok = q_ready(buf))) break;
        for (int st = 0; st < min(n, 2); ++st) {
          if (!(ok = full())) break;
          qk(st, buf, slot);
          release(slot);
          next_slot();
        }
        if (n <= 2) mma_commit(on, smem_u32(&sh.q_empty[buf]));
        for (int i = 0; ok && i < n; ++i) {
          const int st = i & 1;
          if (!(ok = p_ready(st, 0) && full())) break;
          pv(st, 0, slot, i > 1);
          mma_commit(on, smem_u32(&sh.half_done[st]));
          if (!(ok = p_ready(st, 1))) break;
          pv(st, 1, slot, true);
          release(slot);
          next_slot();
          if (i + 2 < n) {
            if (!(ok = full())) break;
            qk(st, buf, slot);
            release(slot);
            next_slot();
            if (i + 3 == n) mma_commit(on, smem_u32(&sh.q_empty[buf]));
          } else {
            mma_commit(on, smem_u32(&sh.o_final[st]));
          }
          p_phase ^= 1u << st;
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
    const int st = (warp - kSoftmaxWarp) >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // TMEM lane of the warp's first row
    const uint32_t tS = tmem + lanes + st * 128, tO = tmem + lanes + 256;
    const uint64_t scale2 = pack2(__float_as_uint(a.scale_log2), __float_as_uint(a.scale_log2));
    const uint64_t one2 = pack2(0x3f800000u, 0x3f800000u);
    int ring0 = 0, tiles0 = 0;                 // ring position, paged tiles before the segment
    uint32_t s_phase = 0, h_phase = 0, o_phase = 0, meet_phase = 0;
    bool ok = true;
    auto meet = [&]() {   // of both streams
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.meet));
      const bool r = pwait_warp(&sh.meet, meet_phase, &sh.abort);
      meet_phase ^= 1;
      return r;
    };
    for (int at = 0; ok; ++at) {
      const Seg* sp = segment(at);
      if (!sp || sp->kind < 0) break;
      const Seg s = *sp;
      done_with(at);
      const int steps = s.steps(st);
      const int rt = s.rt + (s.pair ? st : 0);
      const int rows = min(kTile, a.rows[s.kind] - rt * kTile);
      const bool paged = a.cache[s.kind].page_table != nullptr;
      const bool live = (warp & 3) * 32 < rows;           // the warp has rows
      const int t_row = s.kind ? (rt * kTile + row) % a.w : 0;   // window row of this row
      float m = -INFINITY;
      uint64_t sum = 0;
      for (int step = 0; ok && step < steps; ++step) {
        const int tl = s.tile(st, step), t = s.t0 + tl;
        const bool window = s.kind && t >= s.hist;
        const int valid = s.len - t * kTile;
        // Columns [0, lim) of the tile count.
        const int lim = window ? min(a.w, t_row + 1) - (t - s.hist) * kTile : valid;
        bool special = __any_sync(0xffffffffu, lim < kTile);   // columns that do not count
        const unsigned* bad = nullptr;
        if (paged && !window) {
          const int k = (tiles0 + tl) % kMaskRing;
          ok = pwait_warp(&sh.mask_full[k], ((tiles0 + tl) / kMaskRing) & 1, &sh.abort);
          if (!ok) break;
          bad = sh.bad[k];
          special |= (bad[0] | bad[1] | bad[2] | bad[3]) != 0;
        }
        ok = pwait_warp(&sh.s_full[st], s_phase, &sh.abort);
        if (!ok) break;
        s_phase ^= 1;
        tc_fence_after();
        auto hand_over = [&](int x) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.p_ready[st][x]));
        };
        // The reference m is a maximum of scores seen before.  It moves only
        // when a row's weights 2^(s - m) of 64 columns add up to more than 2^8
        // (or when it is not set yet), so no maximum is taken and O not scaled
        // for most of them, and a weight never exceeds 2^8.  Masks are the
        // slow path's alone, and its code is there once, for both halves
        // (512 rows x 32768 positions: masks in the fast path 70 us, without
        // 62; the fast path unrolled over the halves 57).
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          if (!special && !__any_sync(0xffffffffu, live && m == -INFINITY)) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              if (x != y) continue;
              if (live) {
                uint32_t x0[32], x1[32], p[32];
                tmem_ld32(tS + y * kHalf, x0);
                tmem_ld32(tS + y * kHalf + 32, x1);
                tc_wait_ld();
                const uint64_t mm = pack2(__float_as_uint(-m), __float_as_uint(-m));
                uint64_t part[2] = {0, 0};
                exp32(x0, scale2, mm, part, p);
                exp32(x1, scale2, mm, part, p + 16);
                const uint64_t all = add2(part[0], part[1]);
                if (__any_sync(0xffffffffu, lo_of(all) + hi_of(all) > kMostWeight)) break;
                sum = add2(sum, all);
                tmem_st32(tS + y * (kHalf / 2), p);
                tc_wait_st();
              }
              hand_over(y);
              x = y + 1;
            }
            if (x == 2) break;
          }
          if (live) {
            const uint32_t tX = tS + x * kHalf, tP = tS + x * (kHalf / 2);
            // 32-column chunks with columns that count for some row
            const int nc = !special ? 2
                                    : __any_sync(0xffffffffu, lim > x * kHalf) +
                                          __any_sync(0xffffffffu, lim > x * kHalf + 32);
            auto load = [&](int c, uint32_t (&v)[32]) {
              tmem_ld32(tX + c * 32, v);
              tc_wait_ld();
              if (special) {
                const int left = lim - x * kHalf - c * 32;
                unsigned dead = left >= 32 ? 0u : left <= 0 ? ~0u : ~0u << left;
                if (bad) dead |= bad[2 * x + c];
                if (__any_sync(0xffffffffu, dead)) mask_bits(v, dead);
              }
            };
            float top = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < nc; ++c) {
              uint32_t v[32];
              load(c, v);
              top = max32(v, top);
            }
            top *= a.scale_log2;
            const bool up = top > m;
            if (__any_sync(0xffffffffu, up)) {
              const float f = up ? ex2(m - top) : 1.f;
              if (up) m = top;
              sum = fma2(sum, pack2(__float_as_uint(f), __float_as_uint(f)), 0);
              if (step > 0 || x > 0) {
                // O is scaled once the product before is complete.  That of
                // an earlier tile is: it was issued before these scores.
                if (x) {
                  ok = pwait_warp(&sh.half_done[st], h_phase, &sh.abort);
                  if (!ok) break;
                  tc_fence_after();
                }
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                  const uint32_t to_o = tO + st * 128 + c * 32;
                  uint32_t o[32];
                  tmem_ld32(to_o, o);
                  tc_wait_ld();
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                  tmem_st32(to_o, o);
                }
              }
            }
            // The scaled score rounded as the maximum was: a weight is at
            // most 1 here, whatever the size of the scores.
            const float ms = m == -INFINITY ? 0.f : -m;
            const uint64_t mm = pack2(__float_as_uint(ms), __float_as_uint(ms));
            uint64_t part[2] = {0, 0};
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              uint32_t v[32], p[16];
              if (c < nc) {
                load(c, v);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  v[i] = __float_as_uint(__fmul_rn(__uint_as_float(v[i]), a.scale_log2));
                exp32(v, one2, mm, part, p);
              } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) p[i] = 0;
              }
              tmem_st16(tP + c * 16, p);   // over scores that are read
            }
            sum = add2(sum, add2(part[0], part[1]));
            tc_wait_st();
          }
          // V rows behind the end hold whatever the cache holds there, NaN
          // included: 0 * NaN must not reach O.
          if (x == 0 && !window && valid < kTile && (!s.pair || st == 0)) {
            const int vat = ring0 + s.v_at(tl);
            ok = pwait_warp(&sh.full[vat % C::SLOTS], (vat / C::SLOTS) & 1, &sh.abort);
            if (!ok) break;
            const uint32_t v = ring + vat % C::SLOTS * C::TILE_BYTES;
            const int log_box = a.log_box[s.kind];
            for (int i = valid * 8 + row; i < kTile * 8; i += 128)
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};\n" ::"r"(
                                 v + v_row<D>(i >> 3, log_box) + (c << (log_box + 7)) + (i & 7) * 16),
                             "r"(0)
                             : "memory");
            fence_proxy_async_smem();
          }
          hand_over(x);
        }
        h_phase ^= 1;
      }
      if (!ok) break;
      ring0 += 2 * s.n;
      if (paged) tiles0 += max(0, min(s.t0 + s.n, s.hist) - s.t0);
      if (steps == 0) continue;
      ok = pwait_warp(&sh.o_final[st], o_phase, &sh.abort);
      if (!ok) break;
      o_phase ^= 1;
      tc_fence_after();
      // Partials: a pair's streams write their rows each; of a single's merged
      // ones, stream B writes the lower 16 rows of each warp.  Of 16 columns
      // lane i % 4 of a row's four lanes has 2 i, 2 i + 1, 8 + 2 i, 9 + 2 i, and
      // keeps them together: a row lies in one piece (its 64-column blocks
      // behind one another), 64 bytes of it per store.
      const int sr = a.slot_rows[s.kind];
      const int streams = a.streams[s.kind];
      const long long slot = (long long)s.slot * streams + (s.pair ? st : 0);
      float* out = a.ws_o[s.kind] + slot * sr * D + (lane & 3) * 4;
      float l = lo_of(sum) + hi_of(sum);
      const int first = (warp & 3) * 32 + (lane >> 2);
      auto put = [&](int r, float* to, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
        if (r < rows) *reinterpret_cast<uint4*>(to + r * D) = make_uint4(x, y, z, w);
      };
      if (s.pair || s.n == 1) {
        if (live) {
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int c = 0; c < D; c += 64) {
              uint32_t o[32];
              tmem_ld_16x64(tO + ((uint32_t)half << 20) + st * 128 + c, o);
              tc_wait_ld();
              const int r = first + half * 16;
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                put(r, out + c + i * 2, o[i], o[i + 1], o[i + 4], o[i + 5]);
                put(r + 8, out + c + i * 2, o[i + 2], o[i + 3], o[i + 6], o[i + 7]);
              }
            }
          }
        }
      } else {
        sh.exchange[st][row] = make_float2(m, l);
        if (!(ok = meet())) break;             // both streams' O, m and l are there
        const float2 y = sh.exchange[st ^ 1][row];
        const float big = fmaxf(m, y.x), ref = big == -INFINITY ? 0.f : big;
        const float f0 = ex2(m - ref), f1 = ex2(y.x - ref);
        m = big;
        l = l * f0 + y.y * f1;
        tc_fence_after();
        if (live) {
          const int r = first + st * 16, from = (lane >> 2) + st * 16;
          const float a0 = __shfl_sync(0xffffffffu, f0, from), a1 = __shfl_sync(0xffffffffu, f1, from);
          const float b0 = __shfl_sync(0xffffffffu, f0, from + 8);
          const float b1 = __shfl_sync(0xffffffffu, f1, from + 8);
#pragma unroll
          for (int c = 0; c < D; c += 64) {
            const uint32_t at_o = tO + ((uint32_t)st << 20) + c;
            uint32_t o[32], z[32];
            tmem_ld_16x64(at_o + st * 128, o);
            tmem_ld_16x64(at_o + (st ^ 1) * 128, z);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(fmaf(__uint_as_float(o[i]), i & 2 ? b0 : a0,
                                          __uint_as_float(z[i]) * (i & 2 ? b1 : a1)));
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              put(r, out + c + i * 2, o[i], o[i + 1], o[i + 4], o[i + 5]);
              put(r + 8, out + c + i * 2, o[i + 2], o[i + 3], o[i + 6], o[i + 7]);
            }
          }
        }
        tc_fence_before();
        if (!(ok = meet())) break;             // read before the next segment writes
      }
      if (row < rows && (s.pair || st == 0)) {
        float2* ml = a.ws_ml[s.kind] + slot * sr + row;
        *ml = make_float2(m, l);
        if (s.whole) ml[streams * sr] = make_float2(-INFINITY, 0.f);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc<512>(tmem);
}

// ---- combine: one thread per four columns of an output row, a row's threads
// side by side

struct CombineArgs {
  PrefixKArgs k;
  __nv_bfloat16* o;
  float* lse;
  int rows;            // b * h_q * w
};

constexpr int kCombineThreads = 256;

constexpr int kPartBatch = 64;
constexpr int kInFlight = 8;

// G groups of threads share a row's partials, so that few rows still spread
// over the SMs and each thread's loads are few.
template <int D, int G>
__global__ void __launch_bounds__(kCombineThreads)
    attn_prefix_combine_kernel(const __grid_constant__ CombineArgs c) {
  constexpr int PIECES = D / 4, ROWS = kCombineThreads / (PIECES * G);
  constexpr int TURNS = kCombineThreads / ROWS;
  // Partials of a batch, by row: first m, l and place of each, then, with
  // nothing-seen ones dropped, weight and place (index of its first four
  // columns in float4s, the family in bit 0).
  __shared__ float2 ml_of[ROWS][kPartBatch + 1];
  __shared__ unsigned at_of[ROWS][kPartBatch + 1];
  __shared__ float weight_of[ROWS][kPartBatch + 1];
  __shared__ float m_of[ROWS], l_of[ROWS], rescale_of[ROWS];
  __shared__ int kept_of[ROWS];
  __shared__ float4 sum_of[G > 1 ? G - 1 : 1][ROWS * PIECES];
  const PrefixKArgs& a = c.k;
  // Finding a batch's partials, neighbouring threads take neighbouring rows
  // (their m and l lie together), adding them up, one row's columns.
  const int turn = threadIdx.x / ROWS, mine = threadIdx.x % ROWS;
  const int piece = threadIdx.x % PIECES, out_row = threadIdx.x / PIECES % ROWS;
  const int group = threadIdx.x / (PIECES * ROWS);
  const int row = blockIdx.x * ROWS + mine;
  const bool have = row < c.rows;
  const int seq = have ? quotient(row, a.hq_w, a.inv_hq_w) : 0;
  const int in_seq = have ? row - seq * a.hq_w : 0;
  const int h = quotient(in_seq, a.gw, a.inv_gw), r = in_seq - h * a.gw;
  const int g = quotient(seq, a.per, a.inv_per);
  griddep_wait();
  griddep_launch_dependents();
  const int2* table = reinterpret_cast<const int2*>(a.plan + kPlanInts);
  const int2 of[2] = {table[g], table[a.count[0] + seq]};
  const bool split = a.plan[0];
  // The row's places in family k: base + (e >> two) * stride + (e & two).
  int n[2], base[2], stride[2], two[2], stream[2], in_tile[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int rr = k ? r : (seq - g * a.per) * a.gw + r, rt = rr / kTile;
    const int pairs = a.row_tiles[k] >> 1, sets = (a.row_tiles[k] + 1) >> 1;
    const bool pair = rt < 2 * pairs;
    in_tile[k] = rr - rt * kTile;
    stream[k] = pair ? rt & 1 : 0;
    if (k == 0 && split) {
      const int np = of[k].y & 0xffff, ns = of[k].y >> 16;
      base[k] = of[k].x + h * (pairs * np + ns) + (pair ? rt >> 1 : pairs * np);
      stride[k] = pair ? pairs : 1;
      two[k] = 0;
      n[k] = pair ? np : ns;
    } else {
      base[k] = of[k].x + (h * of[k].y * sets + (rt >> 1)) * 2;
      stride[k] = sets * 2;
      two[k] = 1;
      n[k] = of[k].y * 2;
    }
    if (!have) n[k] = 0;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < ROWS) {
    m_of[threadIdx.x] = -INFINITY;
    l_of[threadIdx.x] = 0.f;
  }
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const int count = n[0] + n[1];
  for (int i0 = 0;; i0 += kPartBatch) {
    for (int i = turn; i < kPartBatch; i += TURNS) {
      const int e = i0 + i;
      float2 ml = make_float2(-INFINITY, 0.f);
      unsigned at = 0;
      if (e < count) {
        const int k = e < n[1] ? 1 : 0;
        const int x = k ? e : e - n[1];
        const int at_place = base[k] + (x >> two[k]) * stride[k] + (x & two[k]);
        const int slot = at_place * a.streams[k] + stream[k];
        at = ((unsigned)slot * a.slot_rows[k] + in_tile[k]) * (D / 2) + k;
        ml = a.ws_ml[k][(long long)slot * a.slot_rows[k] + in_tile[k]];
      }
      ml_of[mine][i] = ml;
      at_of[mine][i] = at;
    }
    __syncthreads();
    // One warp per row: running maximum, weights, the list without gaps.
    for (int x = warp; x < ROWS; x += kCombineThreads / 32) {
      const float2 p0 = ml_of[x][lane], p1 = ml_of[x][lane + 32];
      const unsigned a0 = at_of[x][lane], a1 = at_of[x][lane + 32];
      const float old = m_of[x];
      float top = fmaxf(old, fmaxf(p0.x, p1.x));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float ref = top == -INFINITY ? 0.f : top;
      // A sum of 0: nothing seen, O may be unwritten.  Not so where it is NaN,
      // whatever the maximum (which leaves NaN scores out): that is kept.
      const bool s0 = p0.y != 0.f, s1 = p1.y != 0.f;
      const float w0 = ex2(p0.x - ref), w1 = ex2(p1.x - ref);
      float sum = (s0 ? w0 * p0.y : 0.f) + (s1 ? w1 * p1.y : 0.f);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      const unsigned b0 = __ballot_sync(0xffffffffu, s0), b1 = __ballot_sync(0xffffffffu, s1);
      const unsigned below = (1u << lane) - 1;
      if (s0) {
        const int to = __popc(b0 & below);
        weight_of[x][to] = w0;
        at_of[x][to] = a0;
      }
      if (s1) {
        const int to = __popc(b0) + __popc(b1 & below);
        weight_of[x][to] = w1;
        at_of[x][to] = a1;
      }
      if (lane == 0) {
        const float f = old == -INFINITY ? 0.f : ex2(old - ref);
        m_of[x] = top;
        l_of[x] = l_of[x] * f + sum;
        rescale_of[x] = f;
        kept_of[x] = __popc(b0) + __popc(b1);
      }
    }
    __syncthreads();
    const float f = rescale_of[out_row];
    acc.x *= f;
    acc.y *= f;
    acc.z *= f;
    acc.w *= f;
    const int kept = kept_of[out_row];
    const float4* from[2] = {reinterpret_cast<const float4*>(a.ws_o[0]) + piece,
                             reinterpret_cast<const float4*>(a.ws_o[1]) + piece};
    for (int i = group * kInFlight; i < kept; i += G * kInFlight) {
      float4 v[kInFlight];
#pragma unroll
      for (int j = 0; j < kInFlight; ++j) {
        v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i + j < kept) {
          const unsigned at = at_of[out_row][i + j];
          v[j] = __ldcg((at & 1 ? from[1] : from[0]) + (at >> 1));
        }
      }
#pragma unroll
      for (int j = 0; j < kInFlight; ++j) {
        const float wt = i + j < kept ? weight_of[out_row][i + j] : 0.f;
        acc.x = fmaf(wt, v[j].x, acc.x);
        acc.y = fmaf(wt, v[j].y, acc.y);
        acc.z = fmaf(wt, v[j].z, acc.z);
        acc.w = fmaf(wt, v[j].w, acc.w);
      }
    }
    if (!__syncthreads_or(count > i0 + kPartBatch)) break;   // also: the batch is read
  }
  if (G > 1) {
    if (group > 0) sum_of[group - 1][threadIdx.x % (PIECES * ROWS)] = acc;
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 0; g < G - 1; ++g) {
      const float4 v = sum_of[g][threadIdx.x];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
  }
  const int to = blockIdx.x * ROWS + out_row;
  if (to >= c.rows) return;
  const float m = m_of[out_row], l = l_of[out_row];
  const float inv = l == 0.f ? 0.f : 1.f / l;
  // The columns' order of the partials.
  uint32_t* out = reinterpret_cast<uint32_t*>(c.o + (long long)to * D) + piece / 4 * 8 + piece % 4;
  out[0] = pack_bf16(acc.x * inv, acc.y * inv);
  out[4] = pack_bf16(acc.z * inv, acc.w * inv);
  if (piece == 0) c.lse[to] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ---- host side

// [outer][h_kv][halves][rows][64] of one cache tensor, in boxes of `halves`
// 64-column halves of box_rows rows.  An axis of stride 0 becomes an axis of
// one element.
bool make_map(CUtensorMap* map, const __nv_bfloat16* base, int d, long long rows, long long heads,
              long long outer, const KvView& kv, int box_rows, int halves) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[5] = {64, (cuuint64_t)rows, (cuuint64_t)(d / 64),
                              (cuuint64_t)(kv.sh ? heads : 1), (cuuint64_t)(kv.sb ? outer : 1)};
  const cuuint64_t strides[4] = {(cuuint64_t)kv.sn * 2, 128,
                                 (cuuint64_t)(kv.sh ? kv.sh : kv.sn) * 2,
                                 (cuuint64_t)(kv.sb ? kv.sb : kv.sn) * 2};
  const cuuint32_t box[5] = {64, (cuuint32_t)box_rows, (cuuint32_t)halves, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<__nv_bfloat16*>(base), dims,
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
  a.inv_grid = 1.f / sms;
  a.inv_per = 1.f / a.per;
  a.inv_gw = 1.f / a.gw;
  a.inv_hq_w = 1.f / a.hq_w;
  size_t at = 0;
  for (int k = 0; k < 2; ++k) {
    // Places on the line: two per segment, a segment per set and chunk.  A
    // range r is at least a CTA's even share of the tiles' cost, and a chunk
    // costs a set more than r - kSegmentCost - kPairCost, or is one tile: so
    // beside one per item there are at most (r + 1) / 6.5 segments per CTA for
    // r up to 33 (chunks of one tile, a pair and a single), fewer beyond.
    static_assert(kPairCost == 8 && kSingleCost == 5 && kSegmentCost == 18, "six segments a CTA");
    a.streams[k] = a.row_tiles[k] > 1 ? 2 : 1;
    const size_t items = (size_t)a.count[k] * a.hkv * ((a.row_tiles[k] + 1) / 2);
    const size_t tiles = (a.n[k] + kTile - 1) / kTile + (k ? a.win_tiles : 0);
    const size_t segs = std::min(items * tiles, items + 6 * (size_t)a.grid);
    const size_t rows = std::max<size_t>(2 * segs, a.grid) * a.streams[k] * a.slot_rows[k];
    lay->o[k] = at;
    at += align256(rows * p.d * sizeof(float));
    lay->ml[k] = at;
    at += align256(rows * sizeof(float2));
  }
  lay->plan = at;
  at += align256((size_t)(kPlanInts + 2 * (p.groups + p.b)) * sizeof(int));
  lay->total = at;
  return a;
}

// The split of prefixes of one length (Walk::search for those on the device):
// the M, from the even share on, whose longest CTA is the shortest, the own
// parts taking equal shares of the CTAs left.  Own parts whose lengths are on
// the device count as 5/8 of the longest they may have: a guess a little above
// lengths spread evenly (the measured batches).  Where most are nearly empty, or
// all full, some CTAs end early.
void host_split(PrefixKArgs& a, bool lengths_given, bool own_given) {
  a.split = a.np = a.ns = a.range = 0;
  const long long tp = (a.n[0] + kTile - 1) / kTile;
  const long long most = (a.n[1] + kTile - 1) / kTile;
  const long long to = (own_given ? (5 * most + 7) / 8 : most) + a.win_tiles;
  const int rt = a.row_tiles[0], pairs = rt / 2, single = rt & 1;
  if (lengths_given || tp == 0 || (long long)a.count[0] * a.hkv * ((rt + 1) / 2) > a.grid) return;
  const long long wp = tp * tile_cost(rt) * a.count[0] * a.hkv;
  const long long wo = to * a.count[1] * a.hkv * tile_cost(a.row_tiles[1]) +
                       (to > 0) * (long long)a.count[1] * a.hkv * ((a.row_tiles[1] + 1) / 2) * kSegmentCost;
  const long long share = (wp + wo + a.grid - 1) / a.grid;
  const long long least = std::max<long long>(16, share);
  long long best = LLONG_MAX;
  for (int i = 0; i <= 128; ++i) {
    const long long m = least + least * i / 64;
    const long long np = pairs ? (tp * kPairCost + m - 1) / m : 0;
    const long long ns = single ? (tp * kSingleCost + m - 1) / m : 0;
    const long long split = a.count[0] * a.hkv * (pairs * np + ns);
    const long long own = a.grid - split;   // CTAs left
    if (own < (wo > 0)) continue;
    const long long longest =
        std::max(m + kSegmentCost, wo > 0 ? (wo + own - 1) / own : 0);
    if (longest >= best) continue;
    best = longest;
    a.split = (int)split;
    a.np = (int)np;
    a.ns = (int)ns;
  }
  if (!a.split) return;
  if (rt <= 2 && on_line_is_shorter(best, share)) {
    a.split = 0;
    return;
  }
  const long long tiles = to * a.count[1] * a.hkv * tile_cost(a.row_tiles[1]);
  a.range = (int)std::max<long long>(kMinRange, tiles / std::max<long long>(1, a.grid - a.split));
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
  CombineArgs c{};
  c.k = k;
  c.o = p.o;
  c.lse = p.lse;
  c.rows = p.b * p.hq * p.w;
  // One group where rows alone fill the SMs twice: four instead take a 7B-shaped
  // step of 896 rows from 25.0 to 20.1 us, and one of 5120 rows from 79 to 84.
  constexpr int kRows = kCombineThreads / (D / 4);
  const int ctas = (c.rows + kRows - 1) / kRows;
  const dim3 block(kCombineThreads);
  if (ctas >= 2 * k.grid)
    e = launch_pdl(attn_prefix_combine_kernel<D, 1>, dim3((unsigned)ctas), block, 0, st, c);
  else
    e = launch_pdl(attn_prefix_combine_kernel<D, 4>,
                   dim3((unsigned)((c.rows + kRows / 4 - 1) / (kRows / 4))), block, 0, st, c);
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
  host_split(a, p.prefix_len != nullptr, p.own_len != nullptr);
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
  a.log_box[0] = a.log_box[1] = 7;
  for (int c = 0; c < 2; ++c)
    if (views[c] && views[c]->page_table)   // the largest power of two that divides page and tile
      for (a.log_box[c] = 4; a.log_box[c] < 7 && views[c]->page_size % (2 << a.log_box[c]) == 0;)
        ++a.log_box[c];
  for (int c = 0; c < 3; ++c) {
    if (!views[c]) continue;
    const KvView& kv = *views[c];
    PrefixCache& pc = a.cache[c];
    const bool paged = kv.page_table != nullptr;
    pc.page_table = kv.page_table;
    pc.pages_per_seq = kv.pages_per_seq;
    pc.num_pages = kv.num_pages;
    pc.runs = paged ? kv.page_size >> a.log_box[c] : 1;
    pc.zh = kv.sh ? 1 : 0;
    pc.zb = kv.sb ? 1 : 0;
    const long long outer = paged ? kv.num_pages : c == 0 ? p.groups : p.b;
    const long long r = paged ? kv.page_size : rows[c];
    const int box = 1 << a.log_box[c ? 1 : 0];
    if (!make_map(&maps.k[c], kv.k, p.d, r, p.hkv, outer, kv, box, 1) ||
        !make_map(&maps.v[c], kv.v, p.d, r, p.hkv, outer, kv, box, p.d / 64))
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
