// Verification attention over a cache held in 4 bits: the kernel (attn_kv4_d64.cu,
// attn_kv4_d128.cu instantiate it; attn_kv4.cu joins the parts).
//
// Mathematics: S = scale q K^T, O = softmax(S) V with K and V from records
// (kv4.cuh), by a running reference m per query row: p = 2^(s - m), l = sum p,
// O = sum p v.  m is not the maximum but a number 8 below the largest score seen
// when it was set; it moves only where a weight would reach 2^15 (weights are f16).
// Weights 2^-33 of the largest still round relative to it, and most tiles need
// no maximum at all.
//
// Both products are formed transposed, with 128 cached positions (or the D
// channels) as the tensor core's M and the query rows of one kv head as its N:
//   S^T [position][row]  = K [position][channel]   Q^T      A in tensor memory
//   O^T [channel][row]  += V^T [channel][position] P^T      A in tensor memory
// A step has 8 to 64 rows to a kv head: as M they would be padded to 128 (40 rows:
// 1024 cycles of tensor core per tile, where the bytes of a tile take 800); as N
// they are padded to the next 16.  And K and V, whose 4-bit codes pass through
// registers anyway, go from there to tensor memory; only Q and P are operands in
// shared memory, whose bandwidth 32 KB tiles of K and V in f16 would take up.
//
// f16 holds every cached value exactly (6 bits, 2^-11 .. 2688), and a q row scaled
// by a power of two.
//
// One persistent CTA per SM.  The tiles of all units (sequence, kv head, block of
// rows) lie on a line that the CTAs share in equal ranges; a CTA's part of a unit
// is a segment, whose O, m and l go to the workspace.  Roles of the 20 warps: 0
// issues the products, 1 (and 3, where rows are gathered) loads records, 2 walks the
// CTA's range and prepares Q, 4-7 take K to tensor memory (a thread has a
// position), 8-11 V (a warp has 32 channels: bytes transposed by ldmatrix), 12-15
// and 16-19 are the softmax of the first and the second half of the rows (a thread
// has a position).
#pragma once

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
  float* ws_o;         // [slot][rows][D], unnormalised, without 2^v_exp
  float2* ws_ml;       // [slot][rows]: reference (log2 units), sum
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
// CTA c of g has the tiles [c total / g, (c + 1) total / g), g <= total.
__device__ __forceinline__ int kv4_start(int c, int total, int g) {
  return (int)((long long)c * total / g);
}
__device__ __forceinline__ int kv4_cta(int tile, int total, int g) {
  return (int)((((long long)tile + 1) * g - 1) / total);
}

#ifdef DUSTIN_KV4_KERNEL

namespace {

__device__ unsigned int g_kv4_attn_flags;

constexpr int kTile = kKv4Tile;
constexpr int kWarps = 20, kThreads = kWarps * 32;
constexpr int kMmaWarp = 0, kLoadWarp = 1, kWalkWarp = 2, kLoadWarp2 = 3, kKWarp = 4, kVWarp = 8,
              kSoftmaxWarp = 12;
constexpr int kSegRing = 4, kDeadRing = 32;
// Tensor memory columns, two buffers of 64 each but O.
constexpr int kColS = 0, kColK = 128, kColV = 256, kColO = 384;

// A reference is set this far below the largest score; weights stay below 2^15.
constexpr float kBelow = 8.f;
constexpr uint32_t kMostWeight = 0x7800;

template <int D>
struct Cfg {
  static constexpr int STAGE = kTile * Rec<D>::BYTES;
  static constexpr int STAGES = D == 128 ? 8 : 12;
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
  unsigned long long k_full[2], v_full[2], s_full[2], s_empty[2], p_full[2], pv_done[2];
  unsigned long long q_full[2], q_empty[2], seg_full[kSegRing], seg_empty[kSegRing];
  unsigned long long dead_full[kDeadRing], meet[2], drain;
  Seg seg[kSegRing];
  alignas(16) unsigned dead[kDeadRing][4]; // positions of a tile that do not count
  float qs[2][kKv4Rows];                   // what S of a row is times, to log2 units
  alignas(16) float4 row_of[8][16];        // per softmax warp: {qs, qs, -m, -m} of two rows
  float exchange[2][2][4][32];            // used in turn: a meeting lies between
  alignas(16) __half vscale[4][2][kTile];  // per V warp: scales of its two groups
  int over[2][4];
  int abort;
  uint32_t tmem;
};

// Read in pieces of 16 and 8 bytes.
static_assert(offsetof(Control, dead) % 16 == 0 && offsetof(Control, row_of) % 16 == 0 &&
                  offsetof(Control, vscale) % 16 == 0,
              "alignment");
static_assert(Cfg<64>::STAGE % 1024 == 0 && Cfg<128>::STAGE % 1024 == 0 && Rec<64>::SK % 8 == 0 &&
                  Rec<128>::SK % 8 == 0 && Rec<64>::V % 16 == 0 && Rec<128>::V % 16 == 0,
              "alignment");

template <int D>
constexpr int kSmem = 2 * Cfg<D>::P + 2 * Cfg<D>::Q + Cfg<D>::STAGES * Cfg<D>::STAGE + (int)sizeof(Control);
static_assert(kSmem<128> <= 232448 && kSmem<64> <= 232448, "shared memory of one CTA");

__device__ __forceinline__ void raise_flag(unsigned f) { atomicOr(&g_kv4_attn_flags, f); }

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
// Waits with the library's limit; gives up when another role has.
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
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(r) : "f"(x));
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

template <int D, int NC, bool GATHER>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kv4_kernel(const __grid_constant__ Kv4KArgs a) {
  using C = Cfg<D>;
  using R = Rec<D>;
  constexpr int N = NC / 2;                // rows of a softmax warp
  constexpr int STAGES = C::STAGES;
  extern __shared__ __align__(1024) unsigned char raw[];
  Control& sh = *reinterpret_cast<Control*>(raw + 2 * C::P + 2 * C::Q + STAGES * C::STAGE);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t p_buf = smem_u32(raw), q_buf = p_buf + 2 * C::P, ring = q_buf + 2 * C::Q;

  if (tid == 0) {
    auto init = [](unsigned long long* bar, int count, int n) {
      for (int i = 0; i < n; ++i) mbar_init(smem_u32(bar + i), count);
    };
    constexpr int kLoaders = GATHER ? 2 : 1;
    init(sh.full, GATHER ? 64 + 2 : 1, STAGES);
    init(sh.empty, 8, STAGES);
    init(sh.k_full, 4, 2);
    init(sh.v_full, 4, 2);
    init(sh.s_full, 1, 2);
    init(sh.s_empty, 8, 2);
    init(sh.p_full, 8, 2);
    init(sh.pv_done, 1, 2);
    init(sh.q_full, 1, 2);
    init(sh.q_empty, 1 + 8, 2);
    init(sh.seg_full, 1, kSegRing);
    init(sh.seg_empty, kLoaders + 1 + 4 + 4 + 8, kSegRing);
    init(sh.dead_full, kLoaders, kDeadRing);
    init(sh.meet, 4, 2);
    init(&sh.drain, 1, 1);
    mbar_fence_init();
    sh.abort = 0;
    for (int i = 0; i < 8; ++i) sh.over[i >> 2][i & 3] = 0;
  }
  if (warp == kMmaWarp) tmem_alloc<512>(smem_u32(&sh.tmem));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tmem = sh.tmem;
  const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // tensor memory lane of the warp's first

  // Segment `at` of the ring, once published; null: given up.
  auto segment = [&](int at) -> const Seg* {
    if (!pwait_warp(&sh.seg_full[at % kSegRing], (at / kSegRing) & 1, &sh.abort)) return nullptr;
    return &sh.seg[at % kSegRing];
  };
  auto done_with = [&](int at) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.seg_empty[at % kSegRing]));
  };
  auto arrive = [&](unsigned long long* bar) {         // once per warp
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(bar));
  };

  if (warp == kWalkWarp) {
    // ------------------------------------------------- the range, and its Q
    Walk walk(a);
    Seg s{};
    for (int at = 0;; ++at) {
      const bool more = walk.next(s);
      if (!pwait_warp(&sh.seg_empty[at % kSegRing], (at / kSegRing & 1) ^ 1, &sh.abort)) break;
      if (!more) s.slot = -1;
      if (lane == 0) {
        sh.seg[at % kSegRing] = s;
        mbar_arrive(smem_u32(&sh.seg_full[at % kSegRing]));
      }
      if (!more) break;
      const int buf = at & 1;
      if (!pwait_warp(&sh.q_empty[buf], (at >> 1 & 1) ^ 1, &sh.abort)) break;
      // A row's lanes scale it by the power of two that takes its largest finite
      // entry to [2^13, 2^14): f16 then has all 8 bits of entries down to 2^-30 of
      // that, and fewer to 2^-37.
      constexpr int L = D / 8, STEP = 32 / L, U = 4;
      const int c = lane % L;
      const __nv_bfloat16* q =
          a.q + (((long long)s.bb * a.hkv + s.h) * a.gw + s.row0) * D + c * 8;
      const uint32_t to = q_buf + buf * C::Q + (c / 8) * (kKv4Rows * 128);
      for (int r0 = lane / L; r0 < NC; r0 += STEP * U) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = r0 + u * STEP;
          v[u] = r < s.rows ? __ldg(reinterpret_cast<const uint4*>(q + (long long)r * D))
                            : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = r0 + u * STEP;
          const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t m = (i & 1 ? w[i / 2] >> 16 : w[i / 2]) & 0x7fffu;
            if (m < 0x7f80u) top = max(top, m);
          }
#pragma unroll
          for (int d = 1; d < L; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
          const int e = top ? min(126, 140 - (int)(top >> 7)) : 0;
          const float up = __int_as_float((e + 127) << 23), down = __int_as_float((127 - e) << 23);
          uint32_t h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            h[i] = pack_f16(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
          if (r < NC) {
            sts128(to + r * 128 + ((c % 8 ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
            if (c == 0) sh.qs[buf][r] = a.scale_log2 * down;
          }
        }
      }
      fence_proxy_async_smem();
      arrive(&sh.q_full[buf]);
    }
    if (blockIdx.x == 0 && a.k_len) walk.table();
  } else if (warp == kLoadWarp && !GATHER) {
    // ------------------------- records, as they lie: one copy per run of them
    int i = 0, filled = 0;
    bool ok = true;
    const int runs = kTile / a.run;
    for (int at = 0; ok; ++at) {
      const Seg* sp = segment(at);
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
        arrive(&sh.dead_full[i % kDeadRing]);
        ok = pwait_warp(&sh.empty[st], (i / STAGES & 1) ^ 1, &sh.abort);
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
  } else if ((warp == kLoadWarp || warp == kLoadWarp2) && GATHER) {
    // ------------------------------------- records one by one, 64 of a tile
    const int half = warp == kLoadWarp2;
    int i = 0;
    bool ok = true;
    for (int at = 0; ok; ++at) {
      const Seg* sp = segment(at);
      ok = sp != nullptr;
      if (!ok || sp->slot < 0) break;
      const Seg s = *sp;
      done_with(at);
      const int* idx = a.idx ? a.idx + (long long)s.bb * a.k : nullptr;
      auto position = [&](int t, int u) -> int {       // -1: behind the end
        const int j = t * kTile + half * 64 + u * 32 + lane;
        if (j >= s.len || t >= s.t0 + s.n) return -1;
        return idx ? __ldg(idx + j) : j;
      };
      int at0 = position(s.t0, 0), at1 = position(s.t0, 1);
      for (int t = s.t0; t < s.t0 + s.n; ++t, ++i) {
        const int st = i % STAGES;
        long long off[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int j = u ? at1 : at0;
          const bool in = t * kTile + half * 64 + u * 32 + lane < s.len;
          off[u] = -1;
          if (in && (j < 0 || j >= a.n)) {
            raise_flag(DUSTIN_DEVFLAG_INDEX_RANGE);
          } else if (in) {
            off[u] = place_of(a.kv, s.bb, s.h, j);
            if (off[u] < 0) raise_flag(DUSTIN_DEVFLAG_PAGE_RANGE);
          }
          const unsigned dead = __ballot_sync(0xffffffffu, off[u] < 0);
          if (lane == 0) sh.dead[i % kDeadRing][half * 2 + u] = dead;
        }
        at0 = position(t + 1, 0);
        at1 = position(t + 1, 1);
        arrive(&sh.dead_full[i % kDeadRing]);
        ok = pwait_warp(&sh.empty[st], (i / STAGES & 1) ^ 1, &sh.abort);
        if (!ok) break;
        const uint32_t dst = ring + st * C::STAGE + half * 64 * R::BYTES;
        constexpr int P = R::PIECES;
#pragma unroll
        for (int x0 = 0; x0 < 64 * P; x0 += 32) {
          const int x = x0 + lane, r = x / P, c = x - r * P;
          const long long o0 = __shfl_sync(0xffffffffu, off[0], r & 31);
          const long long o1 = __shfl_sync(0xffffffffu, off[1], r & 31);
          const long long o = r < 32 ? o0 : o1;
          cp_async_16(dst + x * 16, a.kv.data + max(o, 0LL) + c * 16, o < 0 ? 0 : 16);
        }
        const uint32_t bar = smem_u32(&sh.full[st]);
        cp_async_mbar_arrive(bar);
        arrive(&sh.full[st]);
      }
    }
    cp_async_wait<0>();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------- products
    // The whole warp walks, one lane issues.  A tile's scores are asked for
    // before the product of the tile before, so that they are there when the
    // softmax is done with that one.
    constexpr uint32_t kQk = mma_idesc_f16(128, NC, false), kPv = mma_idesc_f16(128, NC, true);
    const uint32_t on = elect_one();
    const uint64_t qd = smem_desc(q_buf, 16, 1024), pd = smem_desc(p_buf, 16, 1024);
    bool ok = true, first = false;         // of the tile whose product is still to come
    int i = 0;
    auto pv = [&](int x, bool fresh) {
      const int buf = x & 1, phase = x >> 1 & 1;
      if (!pwait_warp(&sh.v_full[buf], phase, &sh.abort) ||
          !pwait_warp(&sh.p_full[buf], phase, &sh.abort))
        return false;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        mma_ts(on, tmem + kColO, tmem + kColV + buf * 64 + k * 8,
               pd + ((buf * C::P + k * 2048) >> 4), kPv, !fresh || k > 0);
      mma_commit(on, smem_u32(&sh.pv_done[buf]));
      return true;
    };
    for (int at = 0; ok; ++at) {
      const Seg* sp = segment(at);
      ok = sp != nullptr;
      if (!ok || sp->slot < 0) break;
      const int n = sp->n, qbuf = at & 1;
      done_with(at);
      ok = pwait_warp(&sh.q_full[qbuf], at >> 1 & 1, &sh.abort);
      for (int j = 0; ok && j < n; ++j, ++i) {
        const int buf = i & 1, phase = i >> 1 & 1;
        ok = pwait_warp(&sh.k_full[buf], phase, &sh.abort) &&
             pwait_warp(&sh.s_empty[buf], phase ^ 1, &sh.abort);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ts(on, tmem + kColS + buf * 64, tmem + kColK + buf * 64 + k * 8,
                 qd + ((qbuf * C::Q + (k / 4) * (kKv4Rows * 128) + (k % 4) * 32) >> 4), kQk, k > 0);
        mma_commit(on, smem_u32(&sh.s_full[buf]));
        if (j == n - 1) mma_commit(on, smem_u32(&sh.q_empty[qbuf]));
        if (i > 0) ok = pv(i - 1, first);
        first = j == 0;
      }
    }
    if (ok && i > 0) ok = pv(i - 1, first);
    // The products in flight end before tensor memory is freed.
    mma_commit(on, smem_u32(&sh.drain));
    mbar_wait(smem_u32(&sh.drain), 0, kWaitLimitCycles);
    __syncwarp();
  } else if (warp >= kKWarp && warp < kKWarp + 4) {
    // ------------------------------------------------- K to tensor memory
    int i = 0;
    bool ok = true;
    const uint32_t row = ring + ((warp & 3) * 32 + lane) * R::BYTES;
    for (int at = 0; ok; ++at) {
      const Seg* sp = segment(at);
      if (!sp || sp->slot < 0) break;
      const int n = sp->n;
      done_with(at);
      for (int j = 0; j < n; ++j, ++i) {
        const int st = i % STAGES, buf = i & 1;
        ok = pwait_warp(&sh.full[st], i / STAGES & 1, &sh.abort) &&
             pwait_warp(&sh.s_full[buf], (i >> 1 & 1) ^ 1, &sh.abort);
        if (!ok) break;
        tc_fence_after();
        const uint32_t from = row + st * C::STAGE, to = tmem + lanes + kColK + buf * 64;
        const uint2 sc = lds64(from + R::SK);          // D 64: the first word
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {             // 64 channels, four scales
          const uint32_t four = c ? sc.y : sc.x;
          const uint32_t s01 = e4m3x2_to_f16x2(four), s23 = e4m3x2_to_f16x2(four >> 16);
          const uint32_t s[4] = {__byte_perm(s01, 0, 0x1010), __byte_perm(s01, 0, 0x3232),
                                 __byte_perm(s23, 0, 0x1010), __byte_perm(s23, 0, 0x3232)};
          uint32_t h[32];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint4 v = lds128(from + R::K + c * 32 + x * 16);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint32_t* o = h + x * 16 + y * 4;
              const uint32_t by = s[x * 2 + y / 2];
              o[0] = mul_f16x2(e2m1_to_f16x2<0>(w[y]), by);
              o[1] = mul_f16x2(e2m1_to_f16x2<1>(w[y]), by);
              o[2] = mul_f16x2(e2m1_to_f16x2<2>(w[y]), by);
              o[3] = mul_f16x2(e2m1_to_f16x2<3>(w[y]), by);
            }
          }
          tmem_st32(to + c * 32, h);
        }
        arrive(&sh.empty[st]);
        tc_wait_st();
        tc_fence_before();
        arrive(&sh.k_full[buf]);
      }
    }
  } else if (warp >= kVWarp && warp < kVWarp + 4) {
    // ------------------------------------------------- V to tensor memory
    // Channel c of the warp's groups g = 0, 1 goes to its tensor memory lane
    // 16 g + (c % 2) * 8 + c / 2: a byte holds two channels, and a column of bytes
    // has its lower halves in the first eight lanes.
    const int q = warp & 3;
    const bool live = q * 32 < D;
    int i = 0;
    bool ok = true;
    for (int at = 0; ok; ++at) {
      const Seg* sp = segment(at);
      if (!sp || sp->slot < 0) break;
      const int n = sp->n;
      done_with(at);
      for (int j = 0; j < n; ++j, ++i) {
        const int st = i % STAGES, buf = i & 1;
        ok = pwait_warp(&sh.full[st], i / STAGES & 1, &sh.abort);
        if (!ok) break;
        const uint32_t from = ring + st * C::STAGE;
        if (live) {
          // Scales in f16 by position; positions that do not count have 0, so
          // that no NaN of memory never written meets their weight of 0.
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int p = k * 32 + lane;
            unsigned short two;
            asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(two) : "r"(from + p * R::BYTES + R::SV + q * 2));
            uint32_t s = e4m3x2_to_f16x2(two);
            if (sh.dead[i % kDeadRing][k] >> lane & 1) s = 0;
            sh.vscale[q][0][p] = __ushort_as_half((unsigned short)s);
            sh.vscale[q][1][p] = __ushort_as_half((unsigned short)(s >> 16));
          }
        }
        ok = pwait_warp(&sh.pv_done[buf], (i >> 1 & 1) ^ 1, &sh.abort);
        if (!ok) break;
        tc_fence_after();
        __syncwarp();
        if (live) {
          const uint32_t to = tmem + lanes + kColV + buf * 64;
          const uint32_t scales = smem_u32(&sh.vscale[q][0][0]) + (lane & 3) * 8;
#pragma unroll
          for (int x = 0; x < 4; ++x) {                // 32 positions
            uint32_t w[4];
            ldmatrix_bytes_trans(from + (x * 32 + lane) * R::BYTES + R::V + q * 16, w);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              uint32_t o[8];
#pragma unroll
              for (int y = 0; y < 2; ++y) {            // 16 positions: lane's four
                const uint32_t u = w[2 * y + g];
                const uint2 s = lds64(scales + g * (kTile * 2) + (x * 32 + y * 16) * 2);
                const uint32_t h0 = e2m1_to_f16x2<0>(u), h1 = e2m1_to_f16x2<1>(u);
                const uint32_t h2 = e2m1_to_f16x2<2>(u), h3 = e2m1_to_f16x2<3>(u);
                o[4 * y] = mul_f16x2(__byte_perm(h0, h1, 0x5410), s.x);
                o[4 * y + 1] = mul_f16x2(__byte_perm(h2, h3, 0x5410), s.y);
                o[4 * y + 2] = mul_f16x2(__byte_perm(h0, h1, 0x7632), s.x);
                o[4 * y + 3] = mul_f16x2(__byte_perm(h2, h3, 0x7632), s.y);
              }
              tmem_st_16x16(to + ((uint32_t)g << 20) + x * 16, o);
            }
          }
          tc_wait_st();
        }
        arrive(&sh.empty[st]);
        tc_fence_before();
        arrive(&sh.v_full[buf]);
      }
    }
  } else if (warp >= kSoftmaxWarp) {
    // -------------------------------------------------------------- softmax
    const int wg = (warp - kSoftmaxWarp) >> 2, q = warp & 3, pos = q * 32 + lane;
    const int col0 = wg * N;
    float4* mine = sh.row_of[warp - kSoftmaxWarp];
    const uint32_t row_of = smem_u32(mine);
    const uint32_t tO = tmem + lanes + kColO + col0;
    // The thread's place in P: rows col0 .. col0 + N - 1 of position pos.
    const uint32_t p_row = p_buf + pos * 128;
    int i = 0, votes = 0, turn = 0;
    uint32_t meet_phase = 0;
    bool ok = true;
    auto meet = [&]() {                                // of the warpgroup
      arrive(&sh.meet[wg]);
      const bool r = pwait_warp(&sh.meet[wg], meet_phase, &sh.abort);
      meet_phase ^= 1;
      return r;
    };
    for (int at = 0; ok; ++at) {
      const Seg* sp = segment(at);
      if (!sp || sp->slot < 0) break;
      const int n = sp->n, rows = sp->rows, slot = sp->slot;
      done_with(at);
      ok = pwait_warp(&sh.q_full[at & 1], at >> 1 & 1, &sh.abort);
      if (!ok) break;
      if (lane < N / 2) {
        const float* qs = sh.qs[at & 1] + col0 + 2 * lane;
        mine[lane] = make_float4(qs[0], qs[1], 0.f, 0.f);
      }
      arrive(&sh.q_empty[at & 1]);
      bool fresh = true;                               // no reference yet
      uint64_t l[N / 2];
#pragma unroll
      for (int c = 0; c < N / 2; ++c) l[c] = 0;
      for (int j = 0; j < n; ++j, ++i) {
        const int buf = i & 1, dr = i % kDeadRing;
        ok = pwait_warp(&sh.dead_full[dr], i / kDeadRing & 1, &sh.abort) &&
             pwait_warp(&sh.s_full[buf], i >> 1 & 1, &sh.abort);
        if (!ok) break;
        tc_fence_after();
        const uint4 dead = lds128(smem_u32(sh.dead[dr]));
        bool slow = fresh || (dead.x | dead.y | dead.z | dead.w);
        const uint32_t tS = tmem + lanes + kColS + buf * 64 + col0;
        uint32_t x[N], pk[N / 2];
#pragma unroll
        for (int c = 0; c < N; c += 8) tmem_ld8(tS + c, x + c);
        tc_wait_ld();
        if (!slow) {
          uint32_t most = 0;
#pragma unroll
          for (int c = 0; c < N / 2; ++c) {
            const uint4 r = lds128(row_of + c * 16);
            const uint64_t y = fma2(pack2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])),
                                    pack2(__uint_as_float(r.x), __uint_as_float(r.y)),
                                    pack2(__uint_as_float(r.z), __uint_as_float(r.w)));
            const float e0 = ex2(lo_of(y)), e1 = ex2(hi_of(y));
            x[2 * c] = __float_as_uint(e0);
            x[2 * c + 1] = __float_as_uint(e1);
            pk[c] = pack_f16(e0, e1);
            most = __vmaxu2(most, pk[c]);
          }
          const bool over = (most & 0xffffu) >= kMostWeight || most >> 16 >= kMostWeight;
          const int v = votes++ & 3;
          if (__any_sync(0xffffffffu, over) && lane == 0) *(volatile int*)&sh.over[wg][v] = 1;
          if (q == 0 && lane == 0) *(volatile int*)&sh.over[wg][(v + 2) & 3] = 0;
          ok = meet();
          if (!ok) break;
          slow = *(volatile int*)&sh.over[wg][v] != 0;
        }
        if (slow) {
          // Masks, first tiles and references that move.
          const unsigned word = q == 0 ? dead.x : q == 1 ? dead.y : q == 2 ? dead.z : dead.w;
          const bool gone = word >> lane & 1;
#pragma unroll
          for (int c = 0; c < N; c += 8) tmem_ld8(tS + c, x + c);
          tc_wait_ld();
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const float s = __fmul_rn(__uint_as_float(x[c]), (&mine[c / 2].x)[c & 1]);
            x[c] = __float_as_uint(gone ? -INFINITY : s);
            const float top = warp_max(__uint_as_float(x[c]));
            if (lane == 0) sh.exchange[wg][turn][q][c] = top;
          }
          const float (&from)[4][32] = sh.exchange[wg][turn];
          turn ^= 1;
          ok = meet();
          if (!ok) break;
          // One lane per row: its reference.
          float f = 1.f, minus = 0.f;
          if (lane < N) {
            const float top = fmaxf(fmaxf(from[0][lane], from[1][lane]),
                                    fmaxf(from[2][lane], from[3][lane]));
            const float old = (&mine[lane / 2].z)[lane & 1];
            minus = old;
            if (fresh) {
              minus = top == -INFINITY ? 0.f : kBelow - top;
            } else if (top + old > kBelow) {
              minus = kBelow - top;
              f = ex2(minus - old);
            }
          }
          __syncwarp();
          if (lane < N) (&mine[lane / 2].z)[lane & 1] = minus;
          __syncwarp();
          if (__any_sync(0xffffffffu, minus != minus || f != 1.f)) {
            // O of the tiles before is scaled once their products are complete.
            ok = pwait_warp(&sh.pv_done[(i - 1) & 1], (i - 1) >> 1 & 1, &sh.abort);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < N; c += 8) {
              uint32_t o[8];
              tmem_ld8(tO + c, o);
              tc_wait_ld();
#pragma unroll
              for (int y = 0; y < 8; y += 2) {
                const float f0 = __shfl_sync(0xffffffffu, f, c + y);
                const float f1 = __shfl_sync(0xffffffffu, f, c + y + 1);
                o[y] = __float_as_uint(__uint_as_float(o[y]) * f0);
                o[y + 1] = __float_as_uint(__uint_as_float(o[y + 1]) * f1);
                l[(c + y) / 2] = pack2(lo_of(l[(c + y) / 2]) * f0, hi_of(l[(c + y) / 2]) * f1);
              }
              tmem_st8(tO + c, o);
            }
            tc_wait_st();
          }
          // The scaled score rounded as the maximum was: a weight is at most
          // 2^8 here, whatever the size of the scores.
#pragma unroll
          for (int c = 0; c < N / 2; ++c) {
            const float e0 = ex2(__uint_as_float(x[2 * c]) + mine[c].z);
            const float e1 = ex2(__uint_as_float(x[2 * c + 1]) + mine[c].w);
            x[2 * c] = __float_as_uint(e0);
            x[2 * c + 1] = __float_as_uint(e1);
            pk[c] = pack_f16(e0, e1);
          }
          if ((dead.x & dead.y & dead.z & dead.w) != ~0u) fresh = false;
        }
        tc_fence_before();
        arrive(&sh.s_empty[buf]);
#pragma unroll
        for (int c = 0; c < N / 2; ++c)
          l[c] = add2(l[c], pack2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])));
        ok = pwait_warp(&sh.pv_done[buf], (i >> 1 & 1) ^ 1, &sh.abort);
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < N / 8; ++c)
          sts128(p_row + buf * C::P + (((col0 / 8 + c) ^ (pos & 7)) << 4), pk[4 * c], pk[4 * c + 1],
                 pk[4 * c + 2], pk[4 * c + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        arrive(&sh.p_full[buf]);
      }
      if (!ok) break;
      // The segment's sums over positions: lane c ends with row c's.
      float v[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) v[c] = c < N ? (c & 1 ? hi_of(l[(c % N) / 2]) : lo_of(l[(c % N) / 2])) : 0.f;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int c = 0; c < d; ++c) {
          const float give = lane & d ? v[c] : v[c + d], keep = lane & d ? v[c + d] : v[c];
          v[c] = keep + __shfl_xor_sync(0xffffffffu, give, d);
        }
      const float (&from)[4][32] = sh.exchange[wg][turn];
      sh.exchange[wg][turn][q][lane] = v[0];
      turn ^= 1;
      ok = meet();
      if (!ok) break;
      if (q == 0 && lane < N && col0 + lane < rows) {
        a.ws_ml[(long long)slot * a.rows + col0 + lane] =
            make_float2(-(&mine[lane / 2].z)[lane & 1],
                        from[0][lane] + from[1][lane] + from[2][lane] + from[3][lane]);
      }
      ok = pwait_warp(&sh.pv_done[(i - 1) & 1], (i - 1) >> 1 & 1, &sh.abort);
      if (!ok) break;
      tc_fence_after();
      const int channel = q * 32 + (lane >> 4) * 16 + (lane & 7) * 2 + (lane >> 3 & 1);
      if (q * 32 < D) {
        float* out = a.ws_o + ((long long)slot * a.rows + col0) * D + channel;
#pragma unroll
        for (int c = 0; c < N; c += 8) {
          uint32_t o[8];
          tmem_ld8(tO + c, o);
          tc_wait_ld();
#pragma unroll
          for (int y = 0; y < 8; ++y)
            if (col0 + c + y < rows) out[(c + y) * D] = __uint_as_float(o[y]);
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc<512>(tmem);
}

template <int D, int NC>
cudaError_t run_kv4(const Kv4KArgs& k, bool gather, cudaStream_t st) {
  auto go = [&](auto kern, std::atomic<uint64_t>& done) {
    cudaError_t e = ensure_smem_attr(kern, kSmem<D>, done);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3((unsigned)k.grid), dim3(kThreads), kSmem<D>, st, k);
    if (e == cudaSuccess) note_launches(1);
    return e;
  };
  static std::atomic<uint64_t> done[2];
  return gather ? go(attn_kv4_kernel<D, NC, true>, done[1])
                : go(attn_kv4_kernel<D, NC, false>, done[0]);
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
