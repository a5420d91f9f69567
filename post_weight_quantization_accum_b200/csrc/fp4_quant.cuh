// Quantisation of a lane's values to 4-bit floating point, and the maxima that
// it needs: shared by the quantiser and by the product that quantises its few
// tokens itself, so that both give the same codes.
#pragma once

#include <cfloat>

#include <cuda_fp16.h>

#include "fp4.cuh"

namespace gptq {

// Up to here every CTA reads its group's values itself instead of waiting for
// another kernel's maxima: 128 KB of bf16 take it about two microseconds, a
// second launch and its maxima three.  Groups count by their mean size, and all
// of them for no more than four times as much, in case one has all the rows.
constexpr int64_t kFp4SelfValues = 65536;
inline bool fp4_self_max(int64_t rows, int n, int groups, bool ragged) {
  return ragged ? rows * n <= 4 * kFp4SelfValues && rows * n <= kFp4SelfValues / 2 * groups : rows / groups * n <= kFp4SelfValues;
}

struct QuantArgs {
  const void* X;
  int64_t x_rows, ldx;
  int64_t rows;
  int n;
  const int32_t* row_index;
  const int32_t* offsets;
  int groups;
  int64_t group_rows;  // rows of a group without offsets
  float* tensor_scale;
  uint8_t* packed;
  uint8_t* scales;
  float* deq;
  float* partial;  // amax of (band, split); nullptr: each CTA takes its group's maximum itself
  int splits;      // of a band's columns in `partial`
  int strips;      // a band's rows are quantised by that many CTAs: 1, or 4 of 32 rows
  int given;  // tensor_scale is read, not made
  int vec;  // rows of X start on 32 bytes: 2, on 16: 1, else 0
  int* status;
};

inline QuantArgs fp4_quant_args(const void* X, int x_bf16, int64_t x_rows, int n, int64_t ldx, const int32_t* row_index,
                                int64_t rows, const int32_t* offsets, int groups, int given, float* tensor_scale,
                                int* status) {
  QuantArgs a = {};
  a.X = X;
  a.x_rows = x_rows;
  a.ldx = ldx;
  a.rows = rows;
  a.n = n;
  a.row_index = row_index;
  a.offsets = offsets;
  a.groups = groups;
  a.group_rows = rows / groups;
  a.tensor_scale = tensor_scale;
  a.given = given;
  const uintptr_t at = reinterpret_cast<uintptr_t>(X) | static_cast<uintptr_t>(ldx * (x_bf16 ? 2 : 4));
  a.vec = at % 32 == 0 ? 2 : at % 16 == 0 ? 1 : 0;
  a.status = status;
  return a;
}

// A lane takes 32 bytes of a row, so that a warp's loads are whole lines; a
// block is 1 (nvfp4 of bf16), 2 or 4 (mxfp4 of fp32) neighbouring lanes.
template <bool BF16, bool NV>
struct Fp4Lane {
  static constexpr int kBlock = NV ? 16 : 32;
  static constexpr int kLane = BF16 ? 16 : 8;        // values of a lane
  static constexpr int kLanes = kBlock / kLane;      // lanes of a block
};

__device__ __forceinline__ void load32(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}

// A lane's values as raw words, zeros past the row's end: `left` columns are
// there, and `before` of the row's values stand before them.  VEC: all of
// them, in a 32-byte load (2) or two of 16 (1).  Else in the widest loads that
// the place of the row allows (4-byte words shifted by 16 bits for bf16 on odd
// places), never touching a byte outside the row.
template <bool BF16, int VEC>
__device__ __forceinline__ void load_lane(const char* p, int left, int before, uint32_t (&w)[8]) {
  constexpr int kLane = BF16 ? 16 : 8;
  if (VEC == 2) {
    load32(p, w);
    return;
  }
  const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));
  if (VEC == 1 || (left >= kLane && at % 16 == 0)) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
      w[i] = v.x;
      w[i + 1] = v.y;
      w[i + 2] = v.z;
      w[i + 3] = v.w;
    }
  } else if (left >= kLane && at % 4 == 0) {
    const uint32_t* f = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = f[i];
  } else if (BF16 && left > kLane && before > 0) {
    const uint32_t* f = reinterpret_cast<const uint32_t*>(p - 2);
    uint32_t lo = f[0];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t hi = f[i + 1];
      w[i] = __funnelshift_r(lo, hi, 16);
      lo = hi;
    }
  } else if (BF16) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t lo = 2 * i < left ? h[2 * i] : 0, hi = 2 * i + 1 < left ? h[2 * i + 1] : 0;
      w[i] = lo | hi << 16;
    }
  } else {
    const uint32_t* f = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < left ? f[i] : 0;
  }
}

template <bool BF16>
__device__ __forceinline__ float value(const uint32_t* w, int i) {
  if (!BF16) return __uint_as_float(w[i]);
  return __uint_as_float((i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
}

// Value i of a lane's, in memory.
template <bool BF16>
__device__ __forceinline__ float memory_value(const char* p, int i) {
  if (!BF16) return reinterpret_cast<const float*>(p)[i];
  return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i]) << 16);
}

// Largest magnitude of a lane's values as float bits (from 0x7f800000 on where a
// value is not finite).
template <bool BF16, int WORDS>
__device__ __forceinline__ uint32_t lane_max(const uint32_t (&w)[WORDS]) {
  if (BF16) {  // two at a time, by magnitude (the sign of the result means nothing)
    uint32_t m = w[0];
#pragma unroll
    for (int i = 1; i < WORDS; ++i) asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
    return max(m << 16 & 0x7fff0000u, m & 0x7fff0000u);
  }
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < WORDS; i += 2)
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(__uint_as_float(w[i])), "f"(__uint_as_float(w[i + 1])));
  return __float_as_uint(m) & 0x7fffffffu;
}

// Largest finite magnitude.
template <bool BF16, int WORDS>
__device__ __forceinline__ uint32_t finite_max(const uint32_t (&w)[WORDS]) {
  uint32_t m = lane_max<BF16>(w);
  if (m >= 0x7f800000u) {
    m = 0;
    for (int i = 0; i < (BF16 ? 2 * WORDS : WORDS); ++i) {
      const uint32_t b = __float_as_uint(fabsf(value<BF16>(w, i)));
      if (b < 0x7f800000u) m = max(m, b);
    }
  }
  return m;
}

// Source row of output row r, or -1 (and an error in the status word) where
// the index leaves X.
__device__ __forceinline__ int source_row(const QuantArgs& a, int64_t r) {
  if (a.row_index == nullptr) return static_cast<int>(r);
  const int s = a.row_index[r];
  if (s >= 0 && s < a.x_rows) return s;
  set_status(a.status, GPTQ_ERR_INVALID_ARG);
  return -1;
}

// Largest finite magnitude of a thread's runs of values: kRows of them in flight, given
// by at(i) as pointer (nullptr: none) and columns left.
template <bool BF16, int VEC, int kRows, typename At>
__device__ __forceinline__ uint32_t thread_max(const QuantArgs& a, int first, int step, int count, At at) {
  uint32_t m = 0;
  for (int i0 = first; i0 < count; i0 += kRows * step) {
    uint32_t w[kRows][8];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int i = i0 + u * step;
      int left = 0;
      const char* p = i < count ? at(i, left) : nullptr;
      if (p != nullptr) {
        load_lane<BF16, VEC>(p, left, a.n - left, w[u]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[u][k] = 0;
      }
    }
    uint32_t b = 0;
#pragma unroll
    for (int u = 0; u < kRows; ++u) b = max(b, lane_max<BF16>(w[u]));
    if (b >= 0x7f800000u) {  // something not finite: leave it out
      b = 0;
#pragma unroll
      for (int u = 0; u < kRows; ++u) b = max(b, finite_max<BF16>(w[u]));
    }
    m = max(m, b);
  }
  return m;
}

// Largest finite magnitude of runs of values on any place: at(r, lo, hi) sets
// run r's bytes [lo, hi).  First its whole 16-byte pieces, kPieces at most a run
// (0: `pieces`), 8 of a thread's in flight, then (ENDS) the values before and
// behind them, a thread a run.
template <bool BF16, int kPieces, typename At>
__device__ __forceinline__ uint32_t runs_max(int first, int step, int runs, int pieces, bool ends, At at) {
  constexpr int kFlight = 8;
  const int each = kPieces ? kPieces : pieces, count = runs * each;
  auto up = [](const char* p) { return p + (-reinterpret_cast<uintptr_t>(p) & 15); };
  auto down = [](const char* p) { return p - (reinterpret_cast<uintptr_t>(p) & 15); };
  uint32_t m = 0;
  for (int i0 = first; i0 < count; i0 += kFlight * step) {
    uint32_t w[kFlight][4];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int i = i0 + u * step, r = i / each;
      const char *lo = nullptr, *hi = nullptr;
      if (i < count) at(r, lo, hi);
      const char* p = up(lo) + 16 * (i - r * each);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (p + 16 <= hi) v = *reinterpret_cast<const uint4*>(p);
      w[u][0] = v.x, w[u][1] = v.y, w[u][2] = v.z, w[u][3] = v.w;
    }
    uint32_t b = 0;
#pragma unroll
    for (int u = 0; u < kFlight; ++u) b = max(b, lane_max<BF16>(w[u]));
    if (b >= 0x7f800000u) {  // something not finite: leave it out
      b = 0;
#pragma unroll
      for (int u = 0; u < kFlight; ++u) b = max(b, finite_max<BF16>(w[u]));
    }
    m = max(m, b);
  }
  if (!ends) return m;
  constexpr int kSize = BF16 ? 2 : 4;
  for (int r = first; r < runs; r += step) {
    const char *lo = nullptr, *hi = nullptr;
    at(r, lo, hi);
    const char* head = up(lo) < hi ? up(lo) : hi;
    const char* tail = down(hi) > head ? down(hi) : head;
#pragma unroll
    for (int k = 0; k < 16 / kSize - 1; ++k) {
      float x = 0.0f, y = 0.0f;
      if (lo + k * kSize < head) x = memory_value<BF16>(lo, k);
      if (tail + k * kSize < hi) y = memory_value<BF16>(tail, k);
      const uint32_t bx = __float_as_uint(fabsf(x)), by = __float_as_uint(fabsf(y));
      m = max(m, max(bx < 0x7f800000u ? bx : 0u, by < 0x7f800000u ? by : 0u));
    }
  }
  return m;
}

// Eight values to E2M1, the first in the low bits.
__device__ __forceinline__ uint32_t to_e2m1(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// lo and hi to E4M3 (at most 448), lo in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ float e4m3_value(uint32_t b) {
  return b < 8 ? b * 0.001953125f : __uint_as_float(((b >> 3) + 120) << 23 | (b & 7) << 20);
}

__device__ __forceinline__ float e4m3_to_float(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t k = c & 7;
  const float v = k < 2 ? 0.5f * k : __uint_as_float(((k >> 1) + 126) << 23 | (k & 1) << 22);
  return c & 8 ? -v : v;
}

// E4M3 byte nearest to amax / (6 t), decided on amax against the exact product
// of the border between two neighbours (5 bits) and 6 t (26 bits).
static __device__ __noinline__ uint32_t exact_scale(float amax, float t, uint32_t lo, uint32_t hi) {
  for (uint32_t b = lo; b < hi; ++b) {
    const double border = 0.5 * (double(e4m3_value(b)) + double(e4m3_value(b + 1))) * (6.0 * double(t));
    if (amax < border || (amax == border && b % 2 == 0)) return b;
  }
  return hi;
}

// E2M1 code nearest to x / (s t), on the exact borders.
static __device__ __noinline__ uint32_t exact_code(float x, float s, float t) {
  const double u = double(s) * double(t), a = fabs(double(x));
  uint32_t k = 0;
  while (k < 7) {
    const double border = 0.5 * (double(e2m1_value(k)) + double(e2m1_value(k + 1))) * u;
    if (a < border || (a == border && k % 2 == 0)) break;
    ++k;
  }
  return k | (__float_as_uint(x) >> 31) << 3;
}

// Whether a > border * t, or equal with an odd `below`, on the exact product:
// border has at most 8 bits, so the product is a float and its exact rest, and
// a minus that float is exact where the comparison is near.
__device__ __forceinline__ uint32_t past(float a, float border, float t, uint32_t below) {
  const float near = __fmul_rn(border, t), rest = __fmaf_rn(border, t, -near), d = __fsub_rn(a, near);
  return d > rest || (d == rest && (below & 1));
}
// The border above magnitude code k < 7.
static __constant__ float kE2m1Border[8] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.0f, 0.0f};

constexpr float kBelow = 1.0f - 0x1p-20f, kAbove = 1.0f + 0x1p-20f;

// What a CTA keeps of its group's tensor scale: about 1 / t and 1 / (6 t), a
// rounding each.  Outside [2^-100, 2^100] they, or their products with 1 / s,
// may leave the normal numbers: every decision is then taken in 64 bits.
struct Unit {
  float t, rt, c;
  bool plain;
};
__device__ __forceinline__ Unit unit_of(float t) {
  return {t, __frcp_rn(t), __frcp_rn(__fmul_rn(6.0f, t)), t >= 0x1p-100f && t <= 0x1p100f};
}

__device__ __forceinline__ float rcp_approx(float x) {  // within an ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// (a, b) * (k, k), as one instruction.
__device__ __forceinline__ void mul2(float& a, float& b, float x, float y, float k) {
  asm("{\n\t.reg .b64 p, q;\n\t"
      "mov.b64 p, {%2, %3};\n\t"
      "mov.b64 q, {%4, %4};\n\t"
      "mul.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "=f"(a), "=f"(b)
      : "f"(x), "f"(y), "f"(k));
}

// A lane's part of a block: its codes, and the block's scale byte and s (NaN
// for a block with a value that is not finite: it must not pass for a number,
// and its codes are zero).  p: where the lane's values are in memory, `left` of
// them (the others are zero, and are not read).  Called by whole warps.
template <bool BF16, bool NV>
__device__ __forceinline__ void quantize_lane(const uint32_t (&w)[8], const char* p, int left, const Unit& u,
                                              uint32_t (&codes)[Fp4Lane<BF16, NV>::kLane / 8], uint32_t& byte, float& s) {
  using S = Fp4Lane<BF16, NV>;
  uint32_t m = lane_max<BF16>(w);
#pragma unroll
  for (int d = 1; d < S::kLanes; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (m >= 0x7f800000u) {
    byte = NV ? 0x7f : 0xff;
    s = __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int i = 0; i < S::kLane / 8; ++i) codes[i] = 0;
    return;
  }
  if (!NV) {
    const int lg = m >= 0x00800000u ? int(m >> 23) - 127 : m ? -118 - __clz(m) : -127;
    const int e = max(lg - 2, -127);
    byte = e + 127;
    s = e > -127 ? __uint_as_float(uint32_t(e + 127) << 23) : __uint_as_float(0x00400000u);
    const float inv = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < S::kLane / 8; ++i) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; j += 2) mul2(v[j], v[j + 1], value<BF16>(w, 8 * i + j), value<BF16>(w, 8 * i + j + 1), inv);
      codes[i] = to_e2m1(v);
    }
    return;
  }
  const float amax = __uint_as_float(m);
  // c, two products and a quotient of 24 bits are within 2^-22 of the exact ones
  const uint32_t two = to_e4m3x2(amax * u.c * kBelow, amax * u.c * kAbove);
  byte = two & 0xff;
  if (!u.plain)
    byte = exact_scale(amax, u.t, 0, 126);
  else if (byte != two >> 8)
    byte += past(amax, (e4m3_value(byte) + e4m3_value(byte + 1)) * 3.0f, u.t, byte);  // (neighbours)
  s = e4m3_to_float(byte);
  const float r = rcp_approx(s) * u.rt, r_lo = r * kBelow, r_hi = r * kAbove;
  if (byte == 0) {
#pragma unroll
    for (int i = 0; i < S::kLane / 8; ++i) codes[i] = 0;
    return;
  }
  uint32_t differ[S::kLane / 8];
#pragma unroll
  for (int i = 0; i < S::kLane / 8; ++i) {
    float lo[8], hi[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float x = value<BF16>(w, 8 * i + j), y = value<BF16>(w, 8 * i + j + 1);
      mul2(lo[j], lo[j + 1], x, y, r_lo);
      mul2(hi[j], hi[j + 1], x, y, r_hi);
    }
    codes[i] = to_e2m1(lo);
    differ[i] = codes[i] ^ to_e2m1(hi);
  }
  if (!u.plain) {
#pragma unroll 1
    for (int i = 0; i < S::kLane; ++i) {
      const uint32_t at = 4 * (i % 8), c = exact_code(p == nullptr || i >= left ? 0.0f : memory_value<BF16>(p, i), s, u.t) << at;
      if (i < 8)
        codes[0] = (codes[0] & ~(15u << at)) | c;
      else
        codes[S::kLane / 8 - 1] = (codes[S::kLane / 8 - 1] & ~(15u << at)) | c;
    }
  } else {
    // a border in between (often a tie: bf16 values over a scale made from a
    // bf16 maximum): the code or the next one.  Rolled, with the value read
    // again, as a few lanes of a warp come here.
#pragma unroll
    for (int i = 0; i < S::kLane / 8; ++i) {
#pragma unroll 1
      while (differ[i] != 0) {
        const int at = (__ffs(differ[i]) - 1) & ~3;
        differ[i] &= ~(15u << at);
        const uint32_t k = codes[i] >> at & 7;
        codes[i] += past(fabsf(memory_value<BF16>(p, 8 * i + at / 4)), kE2m1Border[k] * s, u.t, k) << at;
      }
    }
  }
}

}  // namespace gptq
