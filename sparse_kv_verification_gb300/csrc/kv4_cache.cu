// Rows of a cache held in 4 bits: quantised as they are written, and read back.
//
// kv4_write_kernel: of 16 channels x, with y = x * 2^-exp,
//   scale = e4m3_rn(min(max |y| / 6, 448)),  code = e2m1_rn(y / scale),
// ties to even, codes saturated at 6 (both roundings of up to half a step are
// the format's).  kv4_read_kernel: e2m1(code) * e4m3(scale) * 2^exp.
//
// Both decisions are exact.  max |y| / 6 is on the border of two scales only if
// it is a number of 5 bits, which the correctly rounded quotient then is; other
// quotients of an 8-bit number by 6 are 2^-9 of themselves away from it.  y / scale
// is on the border of two codes only if it is one of 0.25, 0.75, 1.25, 1.75, 2.5,
// 3.5, 5; as quotients of 8 bits by 4 bits all others are 1 / 4080 or more away.
// So y times the rounded reciprocal (off by 2^-20 at most below 8) is rounded to
// multiples of 2^-14 first, which puts it back on the border where it belongs
// there, at one addition and one subtraction per value instead of a division.
//
// A lane has 8 channels of a record, two lanes share a scale: 16-byte loads of
// bf16, and a record of D 128 is written (or read) by one warp as 128 + 16 bytes in
// one piece.  Bound by HBM: 4 D bytes of bf16 and one record per row.
#include <algorithm>

#include "dustin.h"
#include "internal.h"
#include "kv4.cuh"

namespace dustin {

namespace {

__device__ unsigned int g_kv4_dev_flags;

__device__ __forceinline__ void raise_flag(unsigned f) { atomicOr(&g_kv4_dev_flags, f); }

constexpr int kThreads = 256;
constexpr int kDeep = 4;         // records a warp has in flight

// Lanes of a record: the first half K, the second V, 8 channels each.
template <int D>
constexpr int kLanes = D / 4;
template <int D>
constexpr int kPerCta = kThreads / kLanes<D> * kDeep;

// 2^e for |e| <= 126.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// The bits of a bf16 pair's larger magnitude, as 15-bit integers: NaN and
// infinity rank above all numbers.
__device__ __forceinline__ uint32_t max_magnitudes(uint32_t a, uint32_t b) {
  return __vmaxu2(a & 0x7fff7fffu, b & 0x7fff7fffu);
}

__device__ __forceinline__ uint32_t e2m1x2(float hi, float lo) {
  uint32_t r;
  asm("{\n .reg .b8 a;\n cvt.rn.satfinite.e2m1x2.f32 a, %1, %2;\n cvt.u32.u8 %0, a;\n}\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A record's place in the lists of a call: sequence, kv head, row.
struct Item {
  int bb, h, t;
};
__device__ __forceinline__ Item item_of(unsigned x, const Kv4Args& a) {
  const unsigned bh = x / (unsigned)a.rows, bb = bh / (unsigned)a.hkv;
  return {(int)bb, (int)(bh - bb * a.hkv), (int)(x - bh * a.rows)};
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const __grid_constant__ Kv4Args a) {
  constexpr int L = kLanes<D>;
  const int lane = threadIdx.x % L, warp = threadIdx.x / L;   // of a record
  const int part = lane >= L / 2, c = lane % (L / 2);         // K or V, its channels 8 c ..
  const KvView& src = a.layer[blockIdx.y].rows;
  const Kv4View& dst = a.layer[blockIdx.y].cache;
  const __nv_bfloat16* from = (part ? src.v : src.k) + c * 8;
  const int exp = part ? dst.v_exp : dst.k_exp;
  griddep_wait();
  griddep_launch_dependents();
  const unsigned first = blockIdx.x * kPerCta<D> + warp;
  uint4 x[kDeep];
  uint8_t* to[kDeep];
#pragma unroll
  for (int u = 0; u < kDeep; ++u) {
    const unsigned i = first + u * (kThreads / L);
    to[u] = nullptr;
    if (i >= a.count) continue;
    const Item it = item_of(i, a);
    if (a.lens && it.t >= __ldg(a.lens + it.bb)) continue;
    const long long j = (a.start ? __ldg(a.start + it.bb) : 0) + (long long)it.t;
    if (j < 0 || j >= a.n) {
      raise_flag(DUSTIN_DEVFLAG_INDEX_RANGE);
      continue;
    }
    const long long s = place_of(src, it.bb, it.h, it.t), d = place_of(dst, it.bb, it.h, (int)j);
    if (s < 0 || d < 0) {
      raise_flag(DUSTIN_DEVFLAG_PAGE_RANGE);
      continue;
    }
    to[u] = const_cast<uint8_t*>(dst.data) + d;
    x[u] = __ldg(reinterpret_cast<const uint4*>(from + s));
  }
#pragma unroll
  for (int u = 0; u < kDeep; ++u) {
    const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
    uint32_t m = max_magnitudes(max_magnitudes(w[0], w[1]), max_magnitudes(w[2], w[3]));
    m = max(m & 0xffffu, m >> 16);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));   // of 16 channels
    if (!to[u]) continue;                             // both lanes of a scale alike
    const bool bad = m >= 0x7f80u;
    const float sixth = __fdiv_rn(__fmul_rn(__uint_as_float(m << 16), pow2(-exp)), 6.f);
    uint32_t scale, two;
    {
      unsigned short h;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %1;\n" : "=h"(h) : "f"(sixth));
      scale = h & 0xffu;
      two = e4m3x2_to_f16x2(h);
    }
    const float step = __half2float(__ushort_as_half((unsigned short)two));
    const float inv = step > 0.f ? __fmul_rn(__frcp_rn(step), pow2(-exp)) : 0.f;
    uint32_t codes = 0;
    constexpr float kGrid = 1.5f * 512.f;             // multiples of 2^-14
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
      const float a0 = copysignf(__fsub_rn(__fmaf_rn(lo, inv, kGrid), kGrid), lo);
      const float a1 = copysignf(__fsub_rn(__fmaf_rn(hi, inv, kGrid), kGrid), hi);
      codes |= e2m1x2(a1, a0) << (8 * i);
    }
    if (bad) codes = 0;
    if (bad) scale = 0x7f;
    uint8_t* rec = to[u];
    *reinterpret_cast<uint32_t*>(rec + part * (D / 2) + c * 4) = codes;
    if (!(lane & 1)) rec[Rec<D>::SK + lane / 2] = (uint8_t)scale;
    if (Rec<D>::SK + L / 2 + lane < Rec<D>::BYTES) rec[Rec<D>::SK + L / 2 + lane] = 0;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const __grid_constant__ Kv4Args a) {
  constexpr int L = kLanes<D>;
  const int lane = threadIdx.x % L, warp = threadIdx.x / L;
  const int part = lane >= L / 2, c = lane % (L / 2);
  const Kv4View& src = a.layer[blockIdx.y].cache;
  const KvView& dst = a.layer[blockIdx.y].rows;
  __nv_bfloat16* base = const_cast<__nv_bfloat16*>(part ? dst.v : dst.k) + c * 8;
  const float unit = pow2(part ? src.v_exp : src.k_exp);
  griddep_wait();
  griddep_launch_dependents();
  const unsigned first = blockIdx.x * kPerCta<D> + warp;
  uint32_t codes[kDeep], scale[kDeep];
  __nv_bfloat16* to[kDeep];
#pragma unroll
  for (int u = 0; u < kDeep; ++u) {
    const unsigned i = first + u * (kThreads / L);
    to[u] = nullptr;
    if (i >= a.count) continue;
    const Item it = item_of(i, a);
    if (a.lens && it.t >= __ldg(a.lens + it.bb)) continue;
    const int j = a.idx ? __ldg(a.idx + (long long)it.bb * a.rows + it.t) : it.t;
    if (j < 0 || j >= a.n) {
      raise_flag(DUSTIN_DEVFLAG_INDEX_RANGE);
      continue;
    }
    const long long s = place_of(src, it.bb, it.h, j), d = place_of(dst, it.bb, it.h, it.t);
    if (s < 0 || d < 0) {
      raise_flag(DUSTIN_DEVFLAG_PAGE_RANGE);
      continue;
    }
    to[u] = base + d;
    codes[u] = __ldg(reinterpret_cast<const uint32_t*>(src.data + s + part * (D / 2) + c * 4));
    scale[u] = __ldg(src.data + s + Rec<D>::SK + lane / 2);
  }
#pragma unroll
  for (int u = 0; u < kDeep; ++u) {
    if (!to[u]) continue;
    const uint32_t s2 = e4m3x2_to_f16x2(scale[u] * 0x101u);
    uint4 out;
    uint32_t* o = &out.x;
    // 6 bits, exact in f16 and in bf16; the exponent shifts it within fp32.
    auto put = [&](int i, uint32_t h2) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      o[i] = pack_bf16(f.x * unit, f.y * unit);
    };
    put(0, mul_f16x2(e2m1_to_f16x2<0>(codes[u]), s2));
    put(1, mul_f16x2(e2m1_to_f16x2<1>(codes[u]), s2));
    put(2, mul_f16x2(e2m1_to_f16x2<2>(codes[u]), s2));
    put(3, mul_f16x2(e2m1_to_f16x2<3>(codes[u]), s2));
    *reinterpret_cast<uint4*>(to[u]) = out;
  }
}

template <typename K>
cudaError_t launch(K kern, const Kv4Args& a, int per_cta, cudaStream_t st) {
  const dim3 grid((a.count + per_cta - 1) / per_cta, a.layers);
  cudaError_t e = launch_pdl(kern, grid, dim3(kThreads), 0, st, a);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4Args& a, int d, cudaStream_t st) {
  return d == 64 ? launch(kv4_write_kernel<64>, a, kPerCta<64>, st)
                 : launch(kv4_write_kernel<128>, a, kPerCta<128>, st);
}

cudaError_t launch_kv4_read(const Kv4Args& a, int d, cudaStream_t st) {
  return d == 64 ? launch(kv4_read_kernel<64>, a, kPerCta<64>, st)
                 : launch(kv4_read_kernel<128>, a, kPerCta<128>, st);
}

cudaError_t take_kv4_flags(unsigned* flags) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv4_dev_flags, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_kv4_dev_flags, &zero, sizeof(zero));
  *flags |= v;
  return e;
}

}  // namespace dustin
