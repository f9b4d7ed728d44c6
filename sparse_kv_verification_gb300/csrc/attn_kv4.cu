// Verification attention over a 4-bit cache: planning, launch, and the kernel that
// joins the parts (attn_kv4.cuh has the attention itself).
//
// The join also adds the window: its w rows are bf16 and few, so each row's
// products with them are formed here in fp32, exactly as they come.  A warp (or
// four, where there are few rows) has a row: per part a reference m_i, a sum l_i and
// O_i, with M the largest of the m_i and of the window's scores s_t,
//   o = (2^v_exp sum_i 2^(m_i - M) O_i + sum_t 2^(s_t - M) V_t) / l,
//   l = sum_i 2^(m_i - M) l_i + sum_t 2^(s_t - M),  lse = ln 2 (M + log2 l),
// in a fixed order.
#include <algorithm>
#include <cmath>

#include "attn_kv4.cuh"

namespace dustin {

namespace {

constexpr int kJoinThreads = 128;
constexpr int kInFlight = 4;

struct JoinArgs {
  Kv4KArgs k;
  __nv_bfloat16* o;
  float* lse;
  KvView win;
  int has_win, w, rows;          // rows: b * h_q * w
  float scale, v_unit;
};

// Weighted sums by a running maximum.
template <int E>
struct Part {
  float m = -INFINITY, l = 0.f, o[E] = {};
  // Before anything of weight 2^to is added.
  __device__ __forceinline__ void raise(float to) {
    if (to > m) {
      const float f = m == -INFINITY ? 0.f : ex2(m - to);
      m = to;
      l = l == 0.f ? 0.f : l * f;            // NaN stays
#pragma unroll
      for (int i = 0; i < E; ++i) o[i] = l == 0.f ? 0.f : o[i] * f;
    }
  }
  __device__ __forceinline__ void add(float weight, float sum, float by, const float (&v)[E]) {
    l = fmaf(weight, sum, l);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(weight * by, v[e], o[e]);
  }
};

template <int E>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, float (&x)[E]) {
  uint32_t w[E / 2];
  if constexpr (E == 4) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x;
    w[1] = v.y;
  } else {
    w[0] = __ldg(reinterpret_cast<const unsigned*>(p));
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
}

// W warps to a row, the loads of kInFlight parts or window positions at a time.
// Measured (72B-shaped, 5120 rows, cold): 8.4 us; 22 with eight parts in flight (126
// registers, two waves) and the window's positions one after another.
template <int D, int W>
__global__ void __launch_bounds__(kJoinThreads, 8)
    attn_kv4_join_kernel(const __grid_constant__ JoinArgs c) {
  constexpr int E = D / 32;      // channels of a lane
  const Kv4KArgs& a = c.k;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, turn = warp % W;
  const int row = blockIdx.x * (kJoinThreads / 32 / W) + warp / W;
  const bool have = row < c.rows;
  const int unit_row = have ? row / a.gw : 0, r = have ? row - unit_row * a.gw : 0;
  const int bb = unit_row / a.hkv, h = unit_row - bb * a.hkv;
  const int block = r / a.rows, in = r - block * a.rows;
  const int hr = a.hkv * a.blocks, unit = h * a.blocks + block;
  griddep_wait();
  griddep_launch_dependents();
  Part<E> part;
  if (have && c.has_win) {
    const int last = r % c.w;                    // window positions 0 .. last
    float q[E];
    load_row<E>(a.q + (long long)row * D + lane * E, q);
    const long long at = (long long)bb * c.win.sb + (long long)h * c.win.sh + lane * E;
    for (int t0 = turn; t0 <= last; t0 += W * kInFlight) {
      float k[kInFlight][E], v[kInFlight][E], s[kInFlight];
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        const int t = min(t0 + i * W, last);     // those past the end are not added
        load_row<E>(c.win.k + at + t * c.win.sn, k[i]);
        load_row<E>(c.win.v + at + t * c.win.sn, v[i]);
      }
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        s[i] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s[i] = fmaf(q[e], k[i][e], s[i]);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        if (t0 + i * W > last) s[i] = -INFINITY;
        // One after the other: scale * log2 e may be no fp32 number.  Rounded, not part of
        // the difference below, or large scores would pass their own maximum.
        s[i] = __fmul_rn(__fmul_rn(s[i], c.scale), kLog2e);
        part.raise(s[i]);
      }
#pragma unroll
      for (int i = 0; i < kInFlight; ++i)
        if (s[i] != -INFINITY) part.add(ex2(s[i] - part.m), 1.f, 1.f, v[i]);
    }
  }
  if (have && a.k > 0) {
    const int tiles = kv4_tiles(kv4_length(a, bb));
    const int total = a.k_len ? a.plan[a.b] : a.b * hr * tiles;
    const int first = (a.k_len ? a.plan[bb] : bb * hr * tiles) + unit * tiles;
    if (tiles > 0) {
      const int g = min(a.grid, total);
      const int c0 = kv4_cta(first, total, g), c1 = kv4_cta(first + tiles - 1, total, g);
      const long long place0 = (long long)(bb * hr + unit + c0) * 2 * a.rows + in;
      const int parts = 2 * (c1 - c0 + 1);       // two streams each
      for (int i0 = turn; i0 < parts; i0 += W * kInFlight) {
        float2 ml[kInFlight];
        float v[kInFlight][E];
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
          const int at = min(i0 + i * W, parts - 1);   // those past the end are not added
          const long long place = place0 + (long long)at * a.rows;
          ml[i] = __ldcg(a.ws_ml + place);
          const float* from = a.ws_o + place * D + lane * E;
          if constexpr (E == 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(from));
            v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
          } else {
            const float2 x = __ldcg(reinterpret_cast<const float2*>(from));
            v[i][0] = x.x, v[i][1] = x.y;
          }
        }
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
          if (i0 + i * W >= parts) ml[i].y = 0.f;
          if (ml[i].y != 0.f) part.raise(ml[i].x);
        }
#pragma unroll
        for (int i = 0; i < kInFlight; ++i)      // a sum of 0: nothing seen, O may be unwritten
          if (ml[i].y != 0.f) part.add(ex2(ml[i].x - part.m), ml[i].y, c.v_unit, v[i]);
      }
    }
  }
  if constexpr (W > 1) {
    __shared__ float2 ml[W];
    __shared__ float os[W][D];
    if (lane == 0) ml[warp] = make_float2(part.m, part.l);
#pragma unroll
    for (int e = 0; e < E; ++e) os[warp][lane * E + e] = part.o[e];
    __syncthreads();
    if (warp) return;
    for (int i = 1; i < W; ++i) {
      if (ml[i].y == 0.f) continue;
      part.raise(ml[i].x);
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = os[i][lane * E + e];
      part.add(ex2(ml[i].x - part.m), ml[i].y, 1.f, v);
    }
  }
  if (!have) return;
  const float inv = part.l == 0.f ? 0.f : 1.f / part.l;
  uint32_t* out = reinterpret_cast<uint32_t*>(c.o + (long long)row * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) out[e / 2] = pack_bf16(part.o[e] * inv, part.o[e + 1] * inv);
  if (lane == 0) c.lse[row] = part.l == 0.f ? -INFINITY : (part.m + log2f(part.l)) * kLn2;
}

template <int D>
cudaError_t join(const JoinArgs& c, cudaStream_t st) {
  // Four warps to a row where rows alone do not fill the SMs.
  constexpr int kPer = kJoinThreads / 32;
  cudaError_t e;
  if (c.rows <= 4 * c.k.grid)
    e = launch_pdl(attn_kv4_join_kernel<D, kPer>, dim3((unsigned)c.rows), dim3(kJoinThreads), 0, st, c);
  else
    e = launch_pdl(attn_kv4_join_kernel<D, 1>, dim3((unsigned)((c.rows + kPer - 1) / kPer)),
                   dim3(kJoinThreads), 0, st, c);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Layout {
  size_t o, ml, plan, total;
};

Kv4KArgs plan(const Kv4AttnArgs& p, int sms, Layout* lay) {
  Kv4KArgs a{};
  a.b = p.b;
  a.hkv = p.hkv;
  a.gw = p.hq / p.hkv * p.w;
  a.n = p.n;
  a.k = p.k;
  a.blocks = (a.gw + kKv4Rows - 1) / kKv4Rows;
  a.rows = (a.gw + a.blocks - 1) / a.blocks;
  a.grid = sms;
  const size_t units = (size_t)p.b * p.hkv * a.blocks;
  const size_t slots = p.k > 0 ? 2 * (units + a.grid) : 0;
  lay->o = 0;
  lay->ml = align256(slots * a.rows * p.d * sizeof(float));
  lay->plan = lay->ml + align256(slots * a.rows * sizeof(float2));
  lay->total = lay->plan + align256((size_t)(p.b + 1) * sizeof(int));
  return a;
}

}  // namespace

size_t attn_kv4_workspace(const Kv4AttnArgs& p, int sms) {
  Layout lay;
  plan(p, sms, &lay);
  return lay.total;
}

cudaError_t launch_attn_kv4(const Kv4AttnArgs& p, int sms, void* ws, cudaStream_t st) {
  Layout lay;
  JoinArgs c{};
  c.k = plan(p, sms, &lay);
  Kv4KArgs& a = c.k;
  char* base = static_cast<char*>(ws);
  a.ws_o = reinterpret_cast<float*>(base + lay.o);
  a.ws_ml = reinterpret_cast<float2*>(base + lay.ml);
  a.plan = reinterpret_cast<int*>(base + lay.plan);
  a.q = p.q;
  a.kv = p.kv;
  a.idx = p.idx;
  a.k_len = p.k_len;
  if (p.k > 0) {
    const int record = p.d == 64 ? Rec<64>::BYTES : Rec<128>::BYTES;
    const bool gather = p.idx || p.kv.sn != record;
    a.run = kKv4Tile;
    if (p.kv.page_table)         // the largest power of two that divides page and tile
      while (p.kv.page_size % a.run) a.run >>= 1;
    // Of 64 bits: the product is an ordinary fp32 number, scale * log2 e need not be.
    a.scale_log2 = (float)std::ldexp((double)p.scale * 1.4426950408889634, p.kv.k_exp);
    cudaError_t e = p.d == 64 ? launch_attn_kv4_d64(a, gather, st) : launch_attn_kv4_d128(a, gather, st);
    if (e != cudaSuccess) return e;
  }
  c.o = p.o;
  c.lse = p.lse;
  c.win = p.win;
  c.has_win = p.has_win;
  c.w = p.w;
  c.rows = p.b * p.hq * p.w;
  c.scale = p.scale;
  c.v_unit = ldexpf(1.f, p.kv.v_exp);
  return p.d == 64 ? join<64>(c, st) : join<128>(c, st);
}

cudaError_t take_attn_kv4_flags(unsigned* flags) {
  cudaError_t e = take_attn_kv4_d64_flags(flags);
  return e != cudaSuccess ? e : take_attn_kv4_d128_flags(flags);
}

}  // namespace dustin
