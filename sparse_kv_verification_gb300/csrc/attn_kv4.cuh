// Verification attention over a cache held in 4 bits: the kernel (attn_kv4_d64.cu,
// attn_kv4_d128.cu instantiate it; attn_kv4.cu joins the parts).
//
// Mathematics: S = scale q K^T, O = softmax(S) V with K and V from records
// (kv4.cuh), by a running reference m per query row: p = 2^(s - m), l = sum p,
// O = sum p v.  m is not the maximum but a number 8 below the largest score seen
// when it was set; it moves only where a weight would pass 2^15 (weights are f16).
// Weights 2^-33 of the largest still round relative to it, and most tiles need
// no maximum at all.
//
// Both products are formed transposed, with 128 cached positions (or the D
// channels) as the tensor core's M and the query rows of one kv head as its N:
//   S^T [position][row]  = K [position][channel]   Q^T      A in tensor memory
//   O^T [channel][row]  += V^T [channel][position] P^T      A in tensor memory
// A step has 8 to 64 rows to a kv head: as M they would be padded to 128 (40 rows:
// 1024 cycles of tensor core per tile, where the bytes of a tile take 800); as N
// they are padded to the next 16, and a product with A in tensor memory takes N / 2
// cycles per 16 deep (measured: 9.2 at N 16, 24.2 at 48; with A in shared memory 39
// and 44).  And K and V, whose 4-bit codes pass through registers anyway, go from
// there to tensor memory; only Q and P are operands in shared memory.
//
// f16 holds every cached value exactly (6 bits, 2^-10 .. 2688), and a q row scaled
// by a power of two.
//
// One persistent CTA per SM.  The tiles of all units (sequence, kv head, block of
// rows) lie on a line that the CTAs share in equal ranges; a CTA's part of a unit
// is a segment.  Its even and odd tiles are two streams, each with an m, l and O of
// its own, so that one's chain (scores, softmax, weights, product) hides the
// other's; the streams' O, m and l go to the workspace.  Roles of the 28 warps: 0
// and 3 issue a stream's products each, 1 loads records, 2 walks the CTA's range;
// 4-11 take the first stream's K and V to tensor memory (K: a thread has a position;
// V: a warp has 32 channels, bytes transposed by ldmatrix), 12-19 the second's;
// 20-23 and 24-27 are a stream's softmax and bring Q.  Where records are gathered
// (idx, or records apart) 4-11 load them and 12-15, 16-19 convert a stream's K and V.
//
// Measured (16 sequences x 32768 positions, 8 kv heads, D 128; bytes alone take 89
// us): 177 us with 40 rows to a kv head, 135 with 8, 241 with 64, 466 with 128 (two
// blocks, each of which reads and converts the cache); D 64 157; 2048 gathered positions
// each 37, of which the join takes 8.  The instance of 49 to 64 rows spills (386 bytes of
// stores; 2.7 % of its warps' instructions are such accesses, 0.1 % at 40 rows): its
// softmax has 64 scores and 48 row factors to hold in 136 registers.  Parts left out of an earlier form of 28 warps (190 us
// whole): without V's conversion 175, without K's 179, without both 164, without the
// softmax 161; without all of these and the products 122: what is left looks like
// the chain of waits between the roles.  How it got here: one stream 251 us; two
// streams 187.  Weights in two buffers, K and V by warps of their own, Q brought by the
// softmax warps and light first tiles read 171, but two waits were missing then (see
// pv_ready and o_done); with a wait at each segment's last tile 194, with o_done 184,
// with the slow path's scores scaled as they are read 177.  (Such changes of rare code
// move the whole by 10 %, either way: the fast path's registers change with it.)
#pragma once

#include <cfloat>
#include <cstddef>

#include "dustin.h"
#include "internal.h"
#include "kv4.cuh"
#include "tcgen05.cuh"

namespace dustin {

constexpr int kKv4Tile = 128;      // positions of a tile
constexpr int kKv4Rows = 64;       // query rows of a block at most

struct Kv4KArgs {
  const __nv_bfloat16* q;
  Kv4View kv;
  const int* idx;
  const int* k_len;
  float* ws_o;         // [slot][stream][rows][D], unnormalised, without 2^v_exp
  float2* ws_ml;       // [slot][stream][rows]: reference (log2 units), sum
  int* plan;           // [b + 1]: where a sequence's tiles start on the line
  int b, hkv, gw, n, k;
  int blocks, rows;    // blocks of rows per kv head, rows of a block
  int grid;
  int run;             // positions of one copy (128: any number)
  float scale_log2;    // with 2^k_exp
};

// ---- the line of tiles, also for the kernel that joins the parts

__device__ __forceinline__ int kv4_length(const Kv4KArgs& a, int bb) {
  return a.k_len ? min(max(__ldg(a.k_len + bb), 0), a.k) : a.k;
}
__device__ __forceinline__ int kv4_tiles(int len) { return (len + kKv4Tile - 1) / kKv4Tile; }
// CTA c of g has the tiles [floor(c total / g), floor((c + 1) total / g)), g <= total:
// with total = q g + r, floor(c total / g) = c q + floor(c r / g), all in 32 bits.
__device__ __forceinline__ int kv4_start(int c, int total, int g) {
  const unsigned q = (unsigned)total / (unsigned)g, r = (unsigned)total - q * g;
  return (int)(c * q + c * r / (unsigned)g);
}
// The last c whose range starts at `tile` or before: the largest with c total < (tile
// + 1) g.  The quotient in fp32 is off by one at most (c < 2^12).
__device__ __forceinline__ int kv4_cta(int tile, int total, int g) {
  const long long x = ((long long)tile + 1) * g;
  int c = (int)__fdividef((float)x, (float)total);
  if ((long long)c * total >= x) --c;
  if ((long long)(c + 1) * total < x) ++c;
  return c;
}

#ifdef DUSTIN_KV4_KERNEL

namespace {

__device__ unsigned int g_kv4_attn_flags;

constexpr int kTile = kKv4Tile;
constexpr int kWarps = 28, kThreads = kWarps * 32;
constexpr int kMmaWarp = 0, kLoadWarp = 1, kWalkWarp = 2, kMmaWarp2 = 3, kCodeWarp = 4,
              kSoftmaxWarp = 20;
// Where records are gathered, half of the warps that convert load them instead.
constexpr int kGatherWarp = 4, kGatherWarps = 8;
constexpr int kSegRing = 4, kDeadRing = 32;
// Tensor memory columns: each stream's S, K, V and O.
constexpr int kColS = 0, kColK = 128, kColV = 256, kColO = 384;

// Registers: a softmax thread holds a tile's scores; the other warps give up what
// it needs beyond the launch's 72.
template <bool GATHER>
struct Split {
  static constexpr int OTHER = 40, LOAD = 40, CODE = GATHER ? 56 : 48, SOFTMAX = 136;
  // In check_register_split's terms: all that give registers up as one warp.
  static constexpr int NT = kThreads, NPW = 1;
  static constexpr int PRODUCER_REGS = 4 * OTHER + (GATHER ? 8 * (LOAD + CODE) : 16 * CODE);
  static constexpr int NCW = 8, CONSUMER_REGS = SOFTMAX;
  static_assert(PRODUCER_REGS + NCW * CONSUMER_REGS <= kWarps * 72, "the launch's registers");
};
template <int R>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(R) : "memory");
}
template <int R>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(R) : "memory");
}

// A reference is set this far below the largest score; weights stay below 2^15.
constexpr float kBelow = 8.f;
constexpr float kMostWeight = 15.f;   // log2

template <int D>
struct Cfg {
  static constexpr int STAGE = kTile * Rec<D>::BYTES;
  static constexpr int PN = 2 /* pv_ready has as many */, STAGES = D == 128 ? 6 : 12;   // buffers of P per stream; tiles in flight
  static constexpr int P = kTile * 128;             // bytes: 64 rows of f16 per position
  static constexpr int Q = D / 64 * kKv4Rows * 128; // 64-channel halves behind one another
};

struct Seg {
  int bb, h, row0, rows;   // sequence, kv head, first row of the block and their number
  int t0, n, len;          // first tile, tiles, positions of the sequence
  int slot;                // -1: no more
};

struct Control {
  unsigned long long full[12], empty[12];
  // Of a stream: K there and S free; each product done.
  unsigned long long qk_ready[2], s_full[2], pv_done[2];
  // A stream's last product of a segment done.  (The softmax may be two products ahead
  // of pv_done, whose parity then says nothing.)
  unsigned long long o_done[2];
  // V and P there, by buffer of P.  With a buffer more than that the softmax may be
  // a tile ahead of V, whose own warps K does not wait for; on one barrier its
  // arrivals would stand in for V's.  On a buffer's, the next are two tiles on, whose
  // scores are asked for after this product.
  unsigned long long pv_ready[2][2];
  unsigned long long q_full[2], q_empty[2], seg_full[kSegRing], seg_empty[kSegRing];
  unsigned long long drain[2];
  Seg seg[kSegRing];
  alignas(16) unsigned dead[kDeadRing][4]; // positions of a tile that do not count
  float qs[2][kKv4Rows];                   // what S of a row is times, to log2 units
  alignas(16) float exchange[2][2][4][kKv4Rows];   // used in turn: a vote lies between
  float minus[2][kKv4Rows];                // -m of a stream's rows, at a segment's end
  alignas(16) __half vscale[8][2][kTile];  // per code warp: V scales of its two groups
  uint32_t tmem;
};

// Read in pieces of 16 and 8 bytes.
static_assert(offsetof(Control, dead) % 16 == 0 && offsetof(Control, exchange) % 16 == 0 &&
                  offsetof(Control, vscale) % 16 == 0 && offsetof(Control, qs) % 8 == 0,
              "alignment");
static_assert(Cfg<64>::STAGE % 1024 == 0 && Cfg<128>::STAGE % 1024 == 0 && Rec<64>::SK % 8 == 0 &&
                  Rec<128>::SK % 8 == 0 && Rec<64>::V % 16 == 0 && Rec<128>::V % 16 == 0,
              "alignment");

template <int D>
constexpr int kSmem = 2 * Cfg<D>::PN * Cfg<D>::P + 2 * Cfg<D>::Q + Cfg<D>::STAGES * Cfg<D>::STAGE + (int)sizeof(Control);
static_assert(kSmem<128> <= 232448 && kSmem<64> <= 232448, "shared memory of one CTA");

__device__ __forceinline__ void raise_flag(unsigned f) { atomicOr(&g_kv4_attn_flags, f); }

// Waits (a whole warp) with the library's limit; the clock is read every 1024 tries
// only, and the code is short: how soon a warp sees that its wait is over sets the
// pace here.
__device__ __forceinline__ bool pwait(unsigned long long* bar, uint32_t parity) {
  static_assert(kWaitLimitCycles == 2000000000LL, "the constant below");
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .u32 n;\n .reg .u64 t, u;\n mov.u64 t, 0;\n"
      "A_%=:\n mov.u32 n, 0;\n"
      "L_%=:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra D_%=;\n"
      " add.u32 n, n, 1;\n setp.lt.u32 q, n, 1024;\n @q bra L_%=;\n"
      " mov.u64 u, %%clock64;\n setp.eq.u64 q, t, 0;\n @q mov.u64 t, u;\n"
      " sub.u64 u, u, t;\n setp.lt.u64 q, u, 2000000000;\n @q bra A_%=;\n"
      "D_%=:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  if (__all_sync(0xffffffffu, ok)) return true;
  raise_flag(DUSTIN_DEVFLAG_WAIT_TIMEOUT);
  return false;
}
// Whether any thread of a warpgroup says so (named barrier `id`).
__device__ __forceinline__ bool vote(int id, bool says) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, %2, 128, q;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)says), "r"(id)
      : "memory");
  return r != 0;
}

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
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// Four 8 x 8 matrices of f16: lane i has two entries of row i / 4 of each, and the
// address of row i % 8 of matrix i / 8.
__device__ __forceinline__ void stmatrix_x4(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
// Two 16 x 16 byte matrices, transposed: of the first (addresses of lanes 0-15)
// lane i gets bytes (rows 4 (i % 4) ..+3, column i / 4) in r[0], column i / 4 + 8
// in r[1]; of the second in r[2], r[3].
__device__ __forceinline__ void ldmatrix_bytes_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Walks the CTA's range of the line (one warp).
struct Walk {
  const Kv4KArgs& a;
  int hr;                        // units of a sequence
  int pos, end;
  int i0, base, t, x;            // 32 sequences at a time: tiles of lane's, sums up to it
  __device__ __forceinline__ void fetch() {
    const int lane = threadIdx.x & 31;
    t = i0 + lane < a.b ? kv4_tiles(kv4_length(a, i0 + lane)) : 0;
    x = t * hr;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
  }
  __device__ explicit Walk(const Kv4KArgs& args) : a(args) {
    hr = a.hkv * a.blocks;
    int total;
    if (a.k_len) {
      total = 0;
      for (int i = threadIdx.x & 31; i < a.b; i += 32) total += kv4_tiles(kv4_length(a, i));
      total = __reduce_add_sync(0xffffffffu, total) * hr;
    } else {
      total = a.b * hr * kv4_tiles(a.k);
    }
    const int g = min(a.grid, total), c = blockIdx.x;
    pos = c < g ? kv4_start(c, total, g) : total;
    end = c < g ? kv4_start(c + 1, total, g) : total;
    i0 = base = 0;
    if (pos < end) {
      if (!a.k_len) {            // straight to the 32 that hold the first tile
        const int per = hr * kv4_tiles(a.k);
        i0 = pos / per & ~31;
        base = i0 * per;
      }
      fetch();
    }
  }
  __device__ __forceinline__ bool next(Seg& s) {
    if (pos >= end) return false;
    unsigned beyond;
    while (!(beyond = __ballot_sync(0xffffffffu, base + x > pos))) {
      base += __shfl_sync(0xffffffffu, x, 31);
      i0 += 32;
      fetch();
    }
    const int at = __ffs(beyond) - 1;
    const int tiles = __shfl_sync(0xffffffffu, t, at);
    const int off = pos - (base + __shfl_sync(0xffffffffu, x, at) - tiles * hr);
    const int unit = off / tiles;
    s.bb = i0 + at;
    s.len = kv4_length(a, s.bb);
    s.t0 = off - unit * tiles;
    s.n = min(tiles - s.t0, end - pos);
    s.h = unit / a.blocks;
    s.row0 = (unit - s.h * a.blocks) * a.rows;
    s.rows = min(a.rows, a.gw - s.row0);
    s.slot = s.bb * hr + unit + blockIdx.x;
    pos += s.n;
    return true;
  }
  // Where each sequence starts, for the kernel that joins the parts.
  __device__ void table() {
    const int lane = threadIdx.x & 31;
    i0 = base = 0;
    for (; i0 < a.b; i0 += 32) {
      fetch();
      if (i0 + lane < a.b) a.plan[i0 + lane] = base + x - t * hr;
      base += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) a.plan[a.b] = base;
  }
};

// Segment `at` of the ring, once published; null: given up.
__device__ __forceinline__ const Seg* segment(Control& sh, int at) {
  if (!pwait(&sh.seg_full[at % kSegRing], (at / kSegRing) & 1)) return nullptr;
  return &sh.seg[at % kSegRing];
}
// One arrival of a warp, after what all its lanes did.
__device__ __forceinline__ void arrive(unsigned long long* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(bar));
}

// All of tensor memory is the CTA's: it starts at 0.
constexpr uint32_t kTmem = 0;

// The products of stream BUF.  A tile's scores are asked for before the product of
// the tile before, as soon as the softmax has read that one's.
template <int D, int NC, int BUF>
__device__ __forceinline__ void products(Control& sh, uint32_t p_buf, uint32_t q_buf) {
  using C = Cfg<D>;
  constexpr uint32_t kQk = mma_idesc_f16(128, NC, false), kPv = mma_idesc_f16(128, NC, true);
  constexpr uint32_t tS = kTmem + kColS + BUF * 64, tK = kTmem + kColK + BUF * 64;
  constexpr uint32_t tV = kTmem + kColV + BUF * 64, tO = kTmem + kColO + BUF * 64;
  const uint32_t on = elect_one();
  const uint64_t qd0 = smem_desc(q_buf, 16, 1024), pd0 = smem_desc(p_buf + BUF * C::PN * C::P, 16, 1024);
  bool ok = true;
  int i = 0, scored = 0, done = 0;         // tiles of the CTA, of the stream
  auto pv = [&](bool fresh) {
    const uint64_t pd = pd0 + (done & (C::PN - 1)) * (C::P >> 4);
    if (!pwait(&sh.pv_ready[BUF][done & 1], done >> 1 & 1)) return false;
    ++done;
    tc_fence_after();
#pragma unroll
    for (int k = 0; k < kTile / 16; ++k)
      mma_ts(on, tO, tV + k * 8, pd + (k * 2048 >> 4), kPv, !fresh || k > 0);
    mma_commit(on, smem_u32(&sh.pv_done[BUF]));
    return true;
  };
  for (int at = 0; ok; ++at) {
    const Seg* sp = segment(sh, at);
    ok = sp != nullptr;
    if (!ok || sp->slot < 0) break;
    const int first = i + ((i ^ BUF) & 1), end = i + sp->n;   // the stream's tiles: first, + 2, ..
    arrive(&sh.seg_empty[at % kSegRing]);
    ok = pwait(&sh.q_full[at & 1], at >> 1 & 1);
    const uint64_t qd = qd0 + ((at & 1) * C::Q >> 4);
    for (int x = first; ok && x < end; x += 2) {
      ok = pwait(&sh.qk_ready[BUF], scored++ & 1);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_ts(on, tS, tK + k * 8, qd + (((k / 4) * (kKv4Rows * 128) + (k % 4) * 32) >> 4), kQk, k > 0);
      mma_commit(on, smem_u32(&sh.s_full[BUF]));
      if (x > first) ok = pv(x == first + 2);
    }
    mma_commit(on, smem_u32(&sh.q_empty[at & 1]));     // also where the stream has none
    if (ok && first < end) {
      ok = pv(first + 2 >= end);
      mma_commit(on, smem_u32(&sh.o_done[BUF]));
    }
    i = end;
  }
  // The products in flight end before tensor memory is freed.
  mma_commit(on, smem_u32(&sh.drain[BUF]));
  mbar_wait(smem_u32(&sh.drain[BUF]), 0, kWaitLimitCycles);
  __syncwarp();
}

template <int D, int NC, bool GATHER>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kv4_kernel(const __grid_constant__ Kv4KArgs a) {
  using C = Cfg<D>;
  using R = Rec<D>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ __align__(1024) unsigned char raw[];
  Control& sh = *reinterpret_cast<Control*>(raw + 2 * C::PN * C::P + 2 * C::Q + STAGES * C::STAGE);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t p_buf = smem_u32(raw), q_buf = p_buf + 2 * C::PN * C::P, ring = q_buf + 2 * C::Q;

  if (tid == 0) {
    auto init = [](unsigned long long* bar, int count, int n) {
      for (int i = 0; i < n; ++i) mbar_init(smem_u32(bar + i), count);
    };
    init(sh.full, GATHER ? 4 * (32 + 1) : 1, STAGES);
    init(sh.empty, GATHER ? 4 : 8, STAGES);
    init(sh.qk_ready, 4 + 1, 2);
    init(sh.pv_ready[0], 4 + 4, 4);
    init(sh.s_full, 1, 2);
    init(sh.pv_done, 1, 2);
    init(sh.o_done, 1, 2);
    init(sh.q_full, 8, 2);
    init(sh.q_empty, 2 + 8, 2);
    init(sh.seg_full, 1, kSegRing);
    init(sh.seg_empty, GATHER ? kGatherWarps + 2 + 8 + 8 : 1 + 2 + 16 + 8, kSegRing);
    init(sh.drain, 1, 2);
    mbar_fence_init();
  }
  if (warp == kMmaWarp) tmem_alloc<512>(smem_u32(&sh.tmem));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  constexpr uint32_t tmem = kTmem;
  const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // tensor memory lane of the warp's first

  auto done_with = [&](int at) { arrive(&sh.seg_empty[at % kSegRing]); };


  // One instruction for a whole warpgroup; the others' stand in their roles, so
  // that the compiler sees what each has.
  if (warp < kCodeWarp) give_registers<Split<GATHER>::OTHER>();

  if (warp == kWalkWarp) {
    // ------------------------------------------------------------ the range
    Walk walk(a);
    Seg s{};
    for (int at = 0;; ++at) {
      const bool more = walk.next(s);
      if (!pwait(&sh.seg_empty[at % kSegRing], (at / kSegRing & 1) ^ 1)) break;
      if (!more) s.slot = -1;
      if (lane == 0) {
        sh.seg[at % kSegRing] = s;
        mbar_arrive(smem_u32(&sh.seg_full[at % kSegRing]));
      }
      if (!more) break;
    }
    if (blockIdx.x == 0 && a.k_len) walk.table();
  } else if (warp == kLoadWarp && !GATHER) {
    // ------------------------- records, as they lie: one copy per run of them
    int i = 0, filled = 0;
    bool ok = true;
    const int runs = kTile / a.run;
    for (int at = 0; ok; ++at) {
      const Seg* sp = segment(sh, at);
      ok = sp != nullptr;
      if (!ok || sp->slot < 0) break;
      const Seg s = *sp;
      done_with(at);
      const uint8_t* data = a.kv.data + (long long)s.h * a.kv.sh;
      auto page_of = [&](int t) -> int {
        const int j = t * kTile + lane * a.run;
        if (lane >= runs || j >= s.len) return 0;
        return __ldg(a.kv.page_table + (long long)s.bb * a.kv.pages_per_seq + j / a.kv.page_size);
      };
      int page = a.kv.page_table ? page_of(s.t0) : 0;
      for (int t = s.t0; t < s.t0 + s.n; ++t, ++i) {
        const int st = i % STAGES;
        const int j = t * kTile + lane * a.run;
        int rows = lane < runs ? min(a.run, max(0, s.len - j)) : 0;
        bool bad = false;
        const uint8_t* src = data + (long long)s.bb * a.kv.sb + (long long)j * R::BYTES;
        if (a.kv.page_table) {
          bad = rows > 0 && (page < 0 || page >= a.kv.num_pages);
          src = data + (long long)page * a.kv.sb + (long long)(j % a.kv.page_size) * R::BYTES;
          if (t + 1 < s.t0 + s.n) page = page_of(t + 1);
          if (bad) {
            rows = 0;
            raise_flag(DUSTIN_DEVFLAG_PAGE_RANGE);
          }
        }
        const unsigned gone = __ballot_sync(0xffffffffu, bad);
        const uint32_t bytes = (uint32_t)__reduce_add_sync(0xffffffffu, rows) * R::BYTES;
        if (lane < 4) {
          const int left = s.len - t * kTile - lane * 32;
          unsigned dead = left >= 32 ? 0u : left <= 0 ? ~0u : ~0u << left;
          if (gone)
            for (int k = 0; k < 32; ++k)
              if (gone >> ((lane * 32 + k) / a.run) & 1) dead |= 1u << k;
          sh.dead[i % kDeadRing][lane] = dead;
        }
        __syncwarp();
        ok = pwait(&sh.empty[st], (i / STAGES & 1) ^ 1);
        if (!ok) break;
        const uint32_t bar = smem_u32(&sh.full[st]);
        if (lane == 0) {
          if (bytes)
            mbar_arrive_expect_tx(bar, bytes);
          else
            mbar_arrive(bar);
        }
        __syncwarp();
        if (rows > 0)
          bulk_g2s(ring + st * C::STAGE + lane * a.run * R::BYTES, src, rows * R::BYTES, bar);
        ++filled;
      }
    }
    // Given up: the copies in flight land before the CTA's memory is reused.
    if (!ok)
      for (int k = max(0, filled - STAGES); k < filled; ++k)
        mbar_wait(smem_u32(&sh.full[k % STAGES]), k / STAGES & 1, kWaitLimitCycles);
  } else if (GATHER && warp >= kGatherWarp && warp < kGatherWarp + kGatherWarps) {
    // ------------- records one by one: four warps a tile, 32 each, in turns
    give_registers<Split<GATHER>::LOAD>();
    const int turn = (warp - kGatherWarp) >> 2, quarter = (warp & 3) * 32;
    int i = 0;
    bool ok = true;
    for (int at = 0; ok; ++at) {
      const Seg* sp = segment(sh, at);
      ok = sp != nullptr;
      if (!ok || sp->slot < 0) break;
      const int bb = sp->bb, h = sp->h, len = sp->len, end = i + sp->n;
      const int from = sp->t0 - i;                     // tile x of the CTA is tile x + from
      done_with(at);
      const int* idx = a.idx ? a.idx + (long long)bb * a.k : nullptr;
      // The lane's position of a tile, fetched one of its tiles ahead.
      auto fetch = [&](int x) -> int {
        const int j = (x + from) * kTile + quarter + lane;
        return x >= end || j >= len ? 0 : idx ? __ldg(idx + j) : j;
      };
      int x = i + ((i ^ turn) & 1);
      int next = fetch(x);
      for (; x < end; x += 2) {
        const int st = x % STAGES, j = next;
        long long off = -1;
        if ((x + from) * kTile + quarter + lane < len) {
          if (j < 0 || j >= a.n) {
            raise_flag(DUSTIN_DEVFLAG_INDEX_RANGE);
          } else {
            off = place_of(a.kv, bb, h, j);
            if (off < 0) raise_flag(DUSTIN_DEVFLAG_PAGE_RANGE);
          }
        }
        const unsigned dead = __ballot_sync(0xffffffffu, off < 0);
        if (lane == 0) sh.dead[x % kDeadRing][warp & 3] = dead;
        next = fetch(x + 2);
        __syncwarp();
        ok = pwait(&sh.empty[st], (x / STAGES & 1) ^ 1);
        if (!ok) break;
        const uint32_t dst = ring + st * C::STAGE + quarter * R::BYTES;
        constexpr int P = R::PIECES;
#pragma unroll
        for (int y = 0; y < P; ++y) {                  // 32 records, a piece per lane
          const int piece = y * 32 + lane, r = piece / P, c = piece - r * P;
          const long long o = __shfl_sync(0xffffffffu, off, r);
          cp_async_16(dst + piece * 16, a.kv.data + max(o, 0LL) + c * 16, o < 0 ? 0 : 16);
        }
        cp_async_mbar_arrive(smem_u32(&sh.full[st]));
        arrive(&sh.full[st]);
      }
      i = end;
    }
    cp_async_wait<0>();
  } else if (warp == kMmaWarp || warp == kMmaWarp2) {
    // ------------------------------------------------ a stream's products
    // A warp per stream: a tile takes it through two waits and 16 products, and the
    // streams do not wait for each other here.
    if (warp == kMmaWarp)
      products<D, NC, 0>(sh, p_buf, q_buf);
    else
      products<D, NC, 1>(sh, p_buf, q_buf);
  } else if (warp >= kCodeWarp && warp < kSoftmaxWarp) {
    // --------------------------- a stream's K, or its V, to tensor memory
    give_registers<Split<GATHER>::CODE>();
    // Two warpgroups per stream, one for K and one for V; where records are gathered
    // one for both.
    const int buf = GATHER ? (warp - kGatherWarp - kGatherWarps) >> 2 : (warp - kCodeWarp) >> 3;
    const int q = warp & 3;
    const bool key = GATHER || !(warp - kCodeWarp & 4), value = GATHER || !key;
    int i = 0;
    bool ok = true;
    const uint32_t to_k = tmem + lanes + kColK + buf * 64, to_v = tmem + lanes + kColV + buf * 64;
    const bool live = q * 32 < D;                      // the warp has channels
    __half (&vscale)[2][kTile] = sh.vscale[buf * 4 + q];
    const uint32_t scales = smem_u32(&vscale[0][0]) + (lane & 3) * 8;
    for (int at = 0; ok; ++at) {
      const Seg* sp = segment(sh, at);
      if (!sp || sp->slot < 0) break;
      const int end = i + sp->n;
      done_with(at);
      for (int x = i + ((i ^ buf) & 1); x < end; x += 2) {
        const int st = x % STAGES, phase = (x >> 1 & 1) ^ 1;
        const uint32_t from = ring + st * C::STAGE;
        ok = pwait(&sh.full[st], x / STAGES & 1);
        if (!ok) break;
        if (key) {
          // K: the thread has a position.
          ok = pwait(&sh.s_full[buf], phase);
          if (!ok) break;
          tc_fence_after();
          const uint32_t row = from + (q * 32 + lane) * R::BYTES;
          const uint2 sc = lds64(row + R::SK);         // D 64: the first word
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {           // 32 channels, two scales
            const uint32_t s01 = e4m3x2_to_f16x2((c < 2 ? sc.x : sc.y) >> (c & 1) * 16);
            const uint32_t s[2] = {__byte_perm(s01, 0, 0x1010), __byte_perm(s01, 0, 0x3232)};
            const uint4 v = lds128(row + R::K + c * 16);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t h[16];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              h[4 * z] = mul_f16x2(e2m1_to_f16x2<0>(w[z]), s[z / 2]);
              h[4 * z + 1] = mul_f16x2(e2m1_to_f16x2<1>(w[z]), s[z / 2]);
              h[4 * z + 2] = mul_f16x2(e2m1_to_f16x2<2>(w[z]), s[z / 2]);
              h[4 * z + 3] = mul_f16x2(e2m1_to_f16x2<3>(w[z]), s[z / 2]);
            }
            tmem_st16(to_k + c * 16, h);
          }
          if (!GATHER) arrive(&sh.empty[st]);
          tc_wait_st();
          tc_fence_before();
          arrive(&sh.qk_ready[buf]);
        }
        if (value) {
          // V: the warp has 32 channels, two groups g.  A byte holds two channels,
          // and a column of bytes has its lower halves in the first eight of 16
          // tensor memory lanes: channel c of a group goes to lane (c % 2) * 8 +
          // c / 2.
          if (live) {
            // Scales in f16 by position; positions that do not count have 0, so
            // that no NaN of memory never written meets their weight of 0.
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int p = k * 32 + lane;
              unsigned short two;
              asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(two) : "r"(from + p * R::BYTES + R::SV + q * 2));
              uint32_t s = e4m3x2_to_f16x2(two);
              if (sh.dead[x % kDeadRing][k] >> lane & 1) s = 0;
              vscale[0][p] = __ushort_as_half((unsigned short)s);
              vscale[1][p] = __ushort_as_half((unsigned short)(s >> 16));
            }
            __syncwarp();
          }
          ok = pwait(&sh.pv_done[buf], phase);
          if (!ok) break;
          tc_fence_after();
          if (live) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {              // 32 positions
              uint32_t w[4];
              ldmatrix_bytes_trans(from + (y * 32 + lane) * R::BYTES + R::V + q * 16, w);
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                uint32_t o[8];
#pragma unroll
                for (int z = 0; z < 2; ++z) {          // 16 positions: lane's four
                  const uint32_t u = w[2 * z + g];
                  const uint2 s = lds64(scales + g * (kTile * 2) + (y * 32 + z * 16) * 2);
                  const uint32_t h0 = e2m1_to_f16x2<0>(u), h1 = e2m1_to_f16x2<1>(u);
                  const uint32_t h2 = e2m1_to_f16x2<2>(u), h3 = e2m1_to_f16x2<3>(u);
                  o[4 * z] = mul_f16x2(__byte_perm(h0, h1, 0x5410), s.x);
                  o[4 * z + 1] = mul_f16x2(__byte_perm(h2, h3, 0x5410), s.y);
                  o[4 * z + 2] = mul_f16x2(__byte_perm(h0, h1, 0x7632), s.x);
                  o[4 * z + 3] = mul_f16x2(__byte_perm(h2, h3, 0x7632), s.y);
                }
                tmem_st_16x16(to_v + ((uint32_t)g << 20) + y * 16, o);
              }
            }
          }
          arrive(&sh.empty[st]);
          tc_wait_st();
          tc_fence_before();
          arrive(&sh.pv_ready[buf][x >> 1 & 1]);
        }
      }
      i = end;
    }
  } else if (warp >= kSoftmaxWarp) {
    // ------------------------------------------------ a stream's softmax
    take_registers<Split<GATHER>::SOFTMAX>();
    // A thread has 4 positions (8 k + lane / 4 of the warp's 32, k = 0 .. 3) and two
    // rows of each 8 (2 (lane % 4), + 1): the rows' factors, references and sums are
    // a quarter of what a position's whole line of rows would take, so that they
    // stay in registers (from shared memory, at 4 cycles per broadcast of 16 bytes,
    // they would take 384 of its cycles per tile: by count, not timed), and the
    // weights leave by stmatrix.
    constexpr int G = NC / 8;                          // groups of 8 rows
    const int buf = (warp - kSoftmaxWarp) >> 2, q = warp & 3;
    const int bar = 1 + buf;                           // named barrier of the warpgroup
    const uint32_t tS = tmem + lanes + kColS + buf * 64, tO = tmem + lanes + kColO + buf * 64;
    const int pos = q * 32 + lane;                     // whose line of P the lane addresses
    const uint32_t p_row0 = p_buf + buf * C::PN * C::P + pos * 128;
    const int col = 2 * (lane & 3);
    // Both streams' warps bring a segment's Q, a segment ahead.  A row's lanes scale it
    // by the power of two that takes its largest finite entry to [2^13, 2^14): f16
    // then has all 8 bits of entries down to 2^-30 of that, and fewer to 2^-37.
    auto bring = [&](int at) -> bool {
      const Seg* sp = segment(sh, at);
      if (!sp) return false;
      if (sp->slot < 0) return true;
      const int have = sp->rows;
      constexpr int L = D / 8, STEP = 8 * 32 / L;      // lanes of a row, rows at a time
      const int c = lane % L, r0 = (warp - kSoftmaxWarp) * (32 / L) + lane / L;
      const __nv_bfloat16* from =
          a.q + (((long long)sp->bb * a.hkv + sp->h) * a.gw + sp->row0) * D + c * 8;
      if (!pwait(&sh.q_empty[at & 1], (at >> 1 & 1) ^ 1)) return false;
      const uint32_t to = q_buf + (at & 1) * C::Q + (c / 8) * (kKv4Rows * 128);
      uint4 v[(NC + STEP - 1) / STEP];
#pragma unroll
      for (int u = 0; u < (NC + STEP - 1) / STEP; ++u) {
        const int r = r0 + u * STEP;
        v[u] = r < have ? __ldg(reinterpret_cast<const uint4*>(from + (long long)r * D)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < (NC + STEP - 1) / STEP; ++u) {
        const int r = r0 + u * STEP;
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        uint32_t top = 0;
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const uint32_t m = (y & 1 ? w[y / 2] >> 16 : w[y / 2]) & 0x7fffu;
          if (m < 0x7f80u) top = max(top, m);
        }
#pragma unroll
        for (int d = 1; d < L; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        const int e = top ? min(126, 140 - (int)(top >> 7)) : 0;
        const float up = __int_as_float((e + 127) << 23), down = __int_as_float((127 - e) << 23);
        uint32_t f[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          f[y] = pack_f16(__uint_as_float(w[y] << 16) * up, __uint_as_float(w[y] & 0xffff0000u) * up);
        if (r < NC) {
          sts128(to + r * 128 + ((c % 8 ^ (r & 7)) << 4), f[0], f[1], f[2], f[3]);
          // Within fp32: 0 times a masked -inf, and infinity times 0, would be NaN.
          if (c == 0) sh.qs[at & 1][r] = fminf(fmaxf(a.scale_log2 * down, 0x1p-126f), 3.4e38f);
        }
      }
      fence_proxy_async_smem();
      arrive(&sh.q_full[at & 1]);
      return true;
    };
    int i = 0, turn = 0, segs = 0;                     // segs: with tiles of the stream
    if (q == 0) arrive(&sh.qk_ready[buf]);             // S is free
    bool ok = bring(0);
    for (int at = 0;; ++at) {
      const Seg* sp = segment(sh, at);
      ok = ok && sp && (sp->slot < 0 || pwait(&sh.q_full[at & 1], at >> 1 & 1));
      // A warp leaves where all of its warpgroup do: after a vote.  Every wait in
      // between has its limit, so every warp gets there.
      if (vote(bar, !ok) || sp->slot < 0) break;
      const int n = sp->n, rows = sp->rows, slot = sp->slot;
      uint64_t qs[G], minus[G], l[G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float2 f = *reinterpret_cast<const float2*>(&sh.qs[at & 1][8 * g + col]);
        qs[g] = pack2(f.x, f.y);
        minus[g] = l[g] = 0;
      }
      arrive(&sh.q_empty[at & 1]);
      ok = bring(at + 1);
      done_with(at);
      bool fresh = true;                               // no reference yet
      int last = -1;                                   // the stream's latest tile
      for (int j = 0; j < n; ++j, ++i) {
        if ((i & 1) != buf) continue;
        const int phase = i >> 1 & 1;
        ok = pwait(&sh.s_full[buf], phase) && ok;
        tc_fence_after();
        const uint4 dead = lds128(smem_u32(sh.dead[i % kDeadRing]));
        uint64_t x[G][4];                              // two rows of position k
        auto load = [&]() {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int g = 0; g < G; g += 2) {
              uint32_t r[8];
              tmem_ld_16x16(tS + ((uint32_t)h << 20) + g * 8, r);
#pragma unroll
              for (int y = 0; y < 4; ++y)
                x[g + y / 2][2 * h + y % 2] = pack2(__uint_as_float(r[2 * y]), __uint_as_float(r[2 * y + 1]));
            }
          tc_wait_ld();
        };
        load();
        // x becomes the weights' exponents.
        float most = -INFINITY;
        bool slow = fresh || (dead.x | dead.y | dead.z | dead.w);
        if (!slow) {
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[g][k] = fma2(x[g][k], qs[g], minus[g]);
              most = max3(most, lo_of(x[g][k]), hi_of(x[g][k]));
            }
        }
        tc_fence_before();
        slow = vote(bar, slow || most > kMostWeight || !ok);
        tc_fence_after();
        if (slow) {
          // Masks, first tiles and references that move.
          const unsigned word = (q == 0 ? dead.x : q == 1 ? dead.y : q == 2 ? dead.z : dead.w) >> (lane >> 2);
          float (&to)[4][kKv4Rows] = sh.exchange[buf][turn];
          turn ^= 1;
          load();
          // Scaled here, one by one, and rounded: a product and a sum of pairs are fused,
          // .rn or not, and half a step of a score past 2^28 takes its weight out of f16.
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[g][k] = pack2(__fmul_rn(lo_of(x[g][k]), lo_of(qs[g])), __fmul_rn(hi_of(x[g][k]), hi_of(qs[g])));
          if (dead.x | dead.y | dead.z | dead.w) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (word >> (8 * k) & 1) {
#pragma unroll
                for (int g = 0; g < G; ++g) x[g][k] = pack2(-INFINITY, -INFINITY);
              }
          }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            float t0 = max3(lo_of(x[g][0]), lo_of(x[g][1]), fmaxf(lo_of(x[g][2]), lo_of(x[g][3])));
            float t1 = max3(hi_of(x[g][0]), hi_of(x[g][1]), fmaxf(hi_of(x[g][2]), hi_of(x[g][3])));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
              t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
            }
            if (lane < 4)
              *reinterpret_cast<float2*>(&to[q][8 * g + col]) = make_float2(t0, t1);
          }
          tc_fence_before();
          if (vote(bar, !ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint64_t f[G];
          bool moves = false;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            // A row without a score above -inf gets the reference of -3.4e38, which any
            // other score moves; its O and sum are 0.
            float top[2] = {-FLT_MAX, -FLT_MAX}, old[2] = {lo_of(minus[g]), hi_of(minus[g])};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float2 t = *reinterpret_cast<const float2*>(&to[w][8 * g + col]);
              top[0] = fmaxf(top[0], t.x);
              top[1] = fmaxf(top[1], t.y);
            }
            float by[2] = {1.f, 1.f};
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              // Rounded down: where neighbouring scores are 16 apart, 8 - top is a tie,
              // and rounded up it would make this very score's exponent 16, past f16.
              const float to_be = __fsub_rd(kBelow, top[y]);
              if (fresh) {
                old[y] = to_be;
              } else if (top[y] + old[y] > kBelow) {
                by[y] = ex2(to_be - old[y]);
                old[y] = to_be;
                moves = true;
              }
            }
            minus[g] = pack2(old[0], old[1]);
            f[g] = pack2(by[0], by[1]);
          }
          if (__any_sync(0xffffffffu, moves)) {
            // O of the tiles before is scaled once their products are complete.
            ok = pwait(&sh.pv_done[buf], phase ^ 1);
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < G; g += 2) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t o[8];
                tmem_ld_16x16(tO + ((uint32_t)h << 20) + g * 8, o);
                tc_wait_ld();
#pragma unroll
                for (int y = 0; y < 8; ++y)
                  o[y] = __float_as_uint(__uint_as_float(o[y]) * (y & 1 ? hi_of(f[g + y / 4]) : lo_of(f[g + y / 4])));
                tmem_st_16x16(tO + ((uint32_t)h << 20) + g * 8, o);
              }
              l[g] = fma2(l[g], f[g], 0);
              l[g + 1] = fma2(l[g + 1], f[g + 1], 0);
            }
            tc_wait_st();
          }
          // As the maximum was rounded, and the reference down: a weight is at most 2^8
          // here, whatever the size of the scores.
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int k = 0; k < 4; ++k) x[g][k] = add2(x[g][k], minus[g]);
          if ((dead.x & dead.y & dead.z & dead.w) != ~0u) fresh = false;
        }
        // All have read S: they have voted since.
        if (q == 0) {
          tc_fence_before();
          arrive(&sh.qk_ready[buf]);
        }
        // This P is free: the product two tiles back in the stream was asked for
        // before these scores, and is done since they are.
        const uint32_t p_row = p_row0 + (phase & (C::PN - 1)) * C::P;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          uint32_t pk[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float e0 = ex2(lo_of(x[g][k])), e1 = ex2(hi_of(x[g][k]));
            l[g] = add2(l[g], pack2(e0, e1));
            pk[k] = pack_f16(e0, e1);
          }
          stmatrix_x4(p_row + ((g ^ (pos & 7)) << 4), pk);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        arrive(&sh.pv_ready[buf][phase]);
        last = i;
      }
      // The rows' sums over positions.
      float (&to)[4][kKv4Rows] = sh.exchange[buf][turn];
      turn ^= 1;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float s0 = lo_of(l[g]), s1 = hi_of(l[g]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          s0 += __shfl_xor_sync(0xffffffffu, s0, d);
          s1 += __shfl_xor_sync(0xffffffffu, s1, d);
        }
        if (lane < 4) {
          *reinterpret_cast<float2*>(&to[q][8 * g + col]) = make_float2(s0, s1);
          if (q == 0) *reinterpret_cast<uint64_t*>(&sh.minus[buf][8 * g + col]) = minus[g];
        }
      }
      if (ok && last >= 0) ok = pwait(&sh.o_done[buf], segs++ & 1);
      tc_fence_after();
      if (vote(bar, !ok)) break;
      const long long place = ((long long)slot * 2 + buf) * a.rows;
      if (q < 2) {
        const int c = q * 32 + lane;
        if (c < rows)
          a.ws_ml[place + c] = make_float2(-sh.minus[buf][c], to[0][c] + to[1][c] + to[2][c] + to[3][c]);
      }
      if (q * 32 < D && last >= 0) {
        // Tensor memory lanes l and l + 8 have neighbouring channels.
        float* out = a.ws_o + (place + col) * D + q * 32 + (lane >> 2) * 2;
#pragma unroll
        for (int g = 0; g < G; g += 2)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t o[8];
            tmem_ld_16x16(tO + ((uint32_t)h << 20) + g * 8, o);
            tc_wait_ld();
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const int c = (g + y) * 8 + z;
                if (c + col < rows)
                  *reinterpret_cast<float2*>(out + c * D + h * 16) =
                      make_float2(__uint_as_float(o[4 * y + z]), __uint_as_float(o[4 * y + 2 + z]));
              }
          }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc<512>(sh.tmem);
}

template <int D, int NC>
cudaError_t run_kv4(const Kv4KArgs& k, bool gather, cudaStream_t st) {
  auto go = [&](auto kern, auto split, std::atomic<uint64_t>& done, std::atomic<int>& split_ok) {
    using S = decltype(split);
    cudaError_t e = ensure_smem_attr(kern, kSmem<D>, done);
    if (e == cudaSuccess) e = check_register_split<S>(kern, split_ok);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3((unsigned)k.grid), dim3(kThreads), kSmem<D>, st, k);
    if (e == cudaSuccess) note_launches(1);
    return e;
  };
  static std::atomic<uint64_t> done[2];
  static std::atomic<int> split_ok[2];
  return gather ? go(attn_kv4_kernel<D, NC, true>, Split<true>(), done[1], split_ok[1])
                : go(attn_kv4_kernel<D, NC, false>, Split<false>(), done[0], split_ok[0]);
}

template <int D>
cudaError_t launch_kv4_rows(const Kv4KArgs& k, bool gather, cudaStream_t st) {
  if (k.rows <= 16) return run_kv4<D, 16>(k, gather, st);
  if (k.rows <= 32) return run_kv4<D, 32>(k, gather, st);
  if (k.rows <= 48) return run_kv4<D, 48>(k, gather, st);
  return run_kv4<D, 64>(k, gather, st);
}

cudaError_t take_kv4_kernel_flags(unsigned* flags) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv4_attn_flags, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_kv4_attn_flags, &zero, sizeof(zero));
  *flags |= v;
  return e;
}

}  // namespace

#endif  // DUSTIN_KV4_KERNEL

// attn_kv4_d64.cu, attn_kv4_d128.cu
cudaError_t launch_attn_kv4_d64(const Kv4KArgs& k, bool gather, cudaStream_t st);
cudaError_t launch_attn_kv4_d128(const Kv4KArgs& k, bool gather, cudaStream_t st);
cudaError_t take_attn_kv4_d64_flags(unsigned* flags);
cudaError_t take_attn_kv4_d128_flags(unsigned* flags);

}  // namespace dustin
