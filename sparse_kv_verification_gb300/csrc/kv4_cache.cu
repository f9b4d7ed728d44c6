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
// one piece.  Traffic is 4 D bytes of bf16 and one record per row, but writing is
// bound by its arithmetic (a prompt's rows: issue 79 %, arithmetic 74 %, DRAM 59 %),
// and gathered reads by the latency of their loads (issue 61 %, DRAM 48 %).
//
// Measured: a prompt's rows written and read back (1375 MB) 243 us, 5.7 TB/s (written
// alone 139, read alone 106); gathered rows read (172 MB) 44 us, 3.9 TB/s; a single row
// written and read back 4.0 us, up to 5 rows of 16 sequences in 16 layers 11: two
// launches each, with the descriptors of 128 layers, 16 KB, as parameters.
#include <algorithm>

#include "dustin.h"
#include "internal.h"
#include "kv4.cuh"

namespace dustin {

namespace {

__device__ unsigned int g_kv4_dev_flags;

__device__ __forceinline__ void raise_flag(unsigned f) { atomicOr(&g_kv4_dev_flags, f); }

constexpr int kThreads = 256;
constexpr int kDeep = 4;         // records of a lane in flight
constexpr int kSteps = 4;        // times that, where the records are one list's

// Lanes of a record: the first half K, the second V, 8 channels each.
template <int D>
constexpr int kLanes = D / 4;
template <int D>
constexpr int kPerCta = kThreads / kLanes<D> * kDeep;

// 2^e for |e| <= 126.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// 1 / x to within one unit in the last place.
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}

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

// The records of a CTA.  Long lists: a piece of one (sequence, kv head)'s, so that
// nothing but the position differs between them; without pages (ROWS) not even that
// has to be looked up.  Short ones (FLAT): of all of them, one after another.
// (All dealt out flat, a prompt of 32749 rows, eight heads and four layers, written
// and read back, took 444 us, most of it quotients and products of strides.)
enum Lists { FLAT, PAGES, ROWS };

// Where a record's bf16 rows and its record lie; false: left out.
template <Lists L>
struct Places {
  const Kv4Args& a;
  const KvView& rows;
  const Kv4View& cache;
  int bb, h, len, start;
  long long rows0, cache0;
  __device__ __forceinline__ explicit Places(const Kv4Args& args)
      : a(args), rows(args.layer[blockIdx.y].rows), cache(args.layer[blockIdx.y].cache) {
    if (L == FLAT) return;
    bb = blockIdx.z / (unsigned)a.hkv;
    h = blockIdx.z - bb * a.hkv;
    len = a.lens ? min(__ldg(a.lens + bb), a.rows) : a.rows;
    start = a.start ? __ldg(a.start + bb) : 0;
    if (L == ROWS) {
      rows0 = bb * rows.sb + h * rows.sh;
      cache0 = bb * cache.sb + h * cache.sh;
    }
  }
  __device__ __forceinline__ bool find(unsigned i, long long& row, long long& rec) const {
    int b = bb, hh = h, t = (int)i, first = start;
    if (L == FLAT) {
      if (i >= a.count) return false;
      const unsigned bh = i / (unsigned)a.rows;
      b = bh / (unsigned)a.hkv;
      hh = bh - b * a.hkv;
      t = i - bh * a.rows;
      if (a.lens && t >= __ldg(a.lens + b)) return false;
      first = a.start ? __ldg(a.start + b) : 0;
    } else if (t >= len) {
      return false;
    }
    const long long j = a.idx ? __ldg(a.idx + (long long)b * a.rows + t) : first + (long long)t;
    if (j < 0 || j >= a.n) {
      raise_flag(DUSTIN_DEVFLAG_INDEX_RANGE);
      return false;
    }
    if (L == ROWS) {
      row = rows0 + t * rows.sn;
      rec = cache0 + j * cache.sn;
      return true;
    }
    row = place_of(rows, b, hh, t);
    rec = place_of(cache, b, hh, (int)j);
    if (row >= 0 && rec >= 0) return true;
    raise_flag(DUSTIN_DEVFLAG_PAGE_RANGE);
    return false;
  }
};

template <int D, Lists LISTS>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const __grid_constant__ Kv4Args a) {
  constexpr int L = kLanes<D>;
  const int lane = threadIdx.x % L, warp = threadIdx.x / L;   // of a record
  const int part = lane >= L / 2, c = lane % (L / 2);         // K or V, its channels 8 c ..
  griddep_wait();
  griddep_launch_dependents();
  const Places<LISTS> places(a);
  const __nv_bfloat16* from = (part ? places.rows.v : places.rows.k) + c * 8;
  const int exp = part ? places.cache.v_exp : places.cache.k_exp;
  uint8_t* data = const_cast<uint8_t*>(places.cache.data);
  unsigned first = blockIdx.x * (kPerCta<D> * (LISTS == FLAT ? 1 : kSteps)) + warp;
#pragma unroll 1
  for (int step = 0; step < (LISTS == FLAT ? 1 : kSteps); ++step, first += kPerCta<D>) {
    uint4 x[kDeep];
    uint8_t* to[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      long long row, rec;
      to[u] = nullptr;
      if (!places.find(first + u * (kThreads / L), row, rec)) continue;
      to[u] = data + rec;
      x[u] = __ldg(reinterpret_cast<const uint4*>(from + row));
    }
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      uint32_t m = max_magnitudes(max_magnitudes(w[0], w[1]), max_magnitudes(w[2], w[3]));
      m = max(m & 0xffffu, m >> 16);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));   // of 16 channels
      if (!to[u]) continue;                             // both lanes of a scale alike
      const bool bad = m >= 0x7f80u;
      // m / 6: the product with the rounded sixth, corrected by its exact remainder,
      // is exact where the quotient is.  (Past 2688 all are one scale.)
      const float y = fminf(__fmul_rn(__uint_as_float(m << 16), pow2(-exp)), 65536.f);
      const float about = __fmul_rn(y, 1.f / 6.f);
      const float sixth = __fmaf_rn(__fmaf_rn(-6.f, about, y), 1.f / 6.f, about);
      uint32_t scale, two;
      {
        unsigned short h;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %1;\n" : "=h"(h) : "f"(sixth));
        scale = h & 0xffu;
        two = e4m3x2_to_f16x2(h);
      }
      const float step = __half2float(__ushort_as_half((unsigned short)two));
      const float inv = step > 0.f ? __fmul_rn(reciprocal(step), pow2(-exp)) : 0.f;
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
}

template <int D, Lists LISTS>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const __grid_constant__ Kv4Args a) {
  constexpr int L = kLanes<D>;
  const int lane = threadIdx.x % L, warp = threadIdx.x / L;
  const int part = lane >= L / 2, c = lane % (L / 2);
  griddep_wait();
  griddep_launch_dependents();
  const Places<LISTS> places(a);
  __nv_bfloat16* base = const_cast<__nv_bfloat16*>(part ? places.rows.v : places.rows.k) + c * 8;
  const float unit = pow2(part ? places.cache.v_exp : places.cache.k_exp);
  const uint8_t* data = places.cache.data;
  unsigned first = blockIdx.x * (kPerCta<D> * (LISTS == FLAT ? 1 : kSteps)) + warp;
#pragma unroll 1
  for (int step = 0; step < (LISTS == FLAT ? 1 : kSteps); ++step, first += kPerCta<D>) {
    uint32_t codes[kDeep], scale[kDeep];
    __nv_bfloat16* to[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      long long row, rec;
      to[u] = nullptr;
      if (!places.find(first + u * (kThreads / L), row, rec)) continue;
      to[u] = base + row;
      codes[u] = __ldg(reinterpret_cast<const uint32_t*>(data + rec + part * (D / 2) + c * 4));
      scale[u] = __ldg(data + rec + Rec<D>::SK + lane / 2);
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
}

template <typename K>
cudaError_t launch(K flat, K pages, K rows, const Kv4Args& a, int per_cta, cudaStream_t st) {
  // A (sequence, kv head)'s list fills CTAs where it has a CTA's records.
  const unsigned lists = a.count / a.rows;
  const int piece = per_cta * kSteps;
  const bool split = a.rows >= piece && lists <= 65535;
  bool paged = false;
  for (int l = 0; l < a.layers; ++l) paged |= a.layer[l].rows.page_table || a.layer[l].cache.page_table;
  const dim3 grid(split ? (a.rows + piece - 1) / piece : (a.count + per_cta - 1) / per_cta, a.layers,
                  split ? lists : 1);
  cudaError_t e = launch_pdl(!split ? flat : paged ? pages : rows, grid, dim3(kThreads), 0, st, a);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4Args& a, int d, cudaStream_t st) {
  return d == 64 ? launch(kv4_write_kernel<64, FLAT>, kv4_write_kernel<64, PAGES>,
                          kv4_write_kernel<64, ROWS>, a, kPerCta<64>, st)
                 : launch(kv4_write_kernel<128, FLAT>, kv4_write_kernel<128, PAGES>,
                          kv4_write_kernel<128, ROWS>, a, kPerCta<128>, st);
}

cudaError_t launch_kv4_read(const Kv4Args& a, int d, cudaStream_t st) {
  return d == 64 ? launch(kv4_read_kernel<64, FLAT>, kv4_read_kernel<64, PAGES>,
                          kv4_read_kernel<64, ROWS>, a, kPerCta<64>, st)
                 : launch(kv4_read_kernel<128, FLAT>, kv4_read_kernel<128, PAGES>,
                          kv4_read_kernel<128, ROWS>, a, kPerCta<128>, st);
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
