// Quantisation to 4-bit floating point (mxfp4, nvfp4).
//
//   mxfp4  blocks of 32: s = 2^(floor(log2 amax) - 2), clamped to 2^[-127, 127]
//   nvfp4  blocks of 16: t = max(RN(amax of the group / 2688), 2^-126),
//          s = E4M3 nearest to amax / (6 t), at most 448
//   code = E2M1 nearest to x / (s t), at most 6, ties to the even code
//
// The quotients are exact: which code is nearest is decided on the real
// numbers, not on rounded ones.  With mxfp4 dividing by s only moves the
// exponent.  With nvfp4 the quotient is bracketed: x r_lo <= x / (s t) <= x r_hi
// with r_lo, r_hi a float or two below and above 1 / (s t), so where both ends
// convert to the same code (all but about 2^-20 of the values) the code is
// certain, and where they do not the exact products b s t of the rounding
// borders b (at most 31 bits) are compared in 64 bits.
//
// Bound by HBM: per value 2 (bf16) or 4 (fp32) bytes in, 1/2 + 1/B out, and 4
// with the dequantised values.  A CTA takes a band of 128 rows x 256 columns,
// a thread a block at a time (its maximum needs no other thread), and the
// band's scale tiles go out whole from shared memory.
#include <algorithm>
#include <cfloat>

#include "fp4.cuh"

namespace gptq {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 256;  // columns of a CTA's tile

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
  int splits;
  int given;  // tensor_scale is read, not made
  int align;  // bytes (32, 16 or 0) that every row of X starts on
  int* status;
};

template <bool BF16, bool NV>
struct Shape {
  static constexpr int kBlock = NV ? 16 : 32;
  static constexpr int kWords = kBlock * (BF16 ? 2 : 4) / 4;
  static constexpr int kCols = kChunk / kBlock;      // blocks across the tile
  static constexpr int kRowsAtOnce = kThreads / kCols;
  static constexpr int kIters = kFp4Band / kRowsAtOnce;
};

__device__ __forceinline__ void load32(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}

__device__ __forceinline__ void store32(void* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// The block's values as raw words, zeros past the row's end.
template <bool BF16, bool NV>
__device__ __forceinline__ void load_block(const QuantArgs& a, int64_t row, int col, uint32_t (&w)[Shape<BF16, NV>::kWords]) {
  using S = Shape<BF16, NV>;
  const int left = a.n - col;
  const char* p = static_cast<const char*>(a.X) + (row * a.ldx + col) * (BF16 ? 2 : 4);
  if (left >= S::kBlock && a.align == 32) {
#pragma unroll
    for (int i = 0; i < S::kWords; i += 8) load32(p + 4 * i, w + i);
  } else if (left >= S::kBlock && a.align == 16) {
#pragma unroll
    for (int i = 0; i < S::kWords; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
      w[i] = v.x;
      w[i + 1] = v.y;
      w[i + 2] = v.z;
      w[i + 3] = v.w;
    }
  } else if (BF16) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < S::kWords; ++i) {
      const uint32_t lo = 2 * i < left ? h[2 * i] : 0, hi = 2 * i + 1 < left ? h[2 * i + 1] : 0;
      w[i] = lo | hi << 16;
    }
  } else {
    const uint32_t* f = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
    for (int i = 0; i < S::kWords; ++i) w[i] = i < left ? f[i] : 0;
  }
}

template <bool BF16>
__device__ __forceinline__ float value(const uint32_t* w, int i) {
  if (!BF16) return __uint_as_float(w[i]);
  return __uint_as_float((i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
}

// Largest magnitude of the block as float bits (an infinity or NaN shows as
// bits >= 0x7f800000, as magnitudes order like their bits).
template <bool BF16, int WORDS>
__device__ __forceinline__ uint32_t block_max(const uint32_t (&w)[WORDS]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < WORDS; ++i) m = BF16 ? __vmaxu2(m, w[i] & 0x7fff7fffu) : max(m, w[i] & 0x7fffffffu);
  return BF16 ? max(m << 16, m & 0xffff0000u) : m;
}

// Largest finite magnitude.
template <bool BF16, int WORDS>
__device__ __forceinline__ uint32_t finite_max(const uint32_t (&w)[WORDS]) {
  uint32_t m = block_max<BF16>(w);
  if (m >= 0x7f800000u) {
    m = 0;
    for (int i = 0; i < (BF16 ? 2 * WORDS : WORDS); ++i) {
      const uint32_t b = __float_as_uint(fabsf(value<BF16>(w, i)));
      if (b < 0x7f800000u) m = max(m, b);
    }
  }
  return m;
}

__device__ __forceinline__ uint32_t cta_max(uint32_t m, uint32_t* s) {
  m = __reduce_max_sync(0xffffffffu, m);
  if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = m;
  __syncthreads();
  m = __reduce_max_sync(0xffffffffu, threadIdx.x % 32 < kThreads / 32 ? s[threadIdx.x % 32] : 0u);
  __syncthreads();
  return m;
}

// Source row of output row r, or -1 (and an error in the status word) where
// the index leaves X.
__device__ __forceinline__ int64_t source_row(const QuantArgs& a, int64_t r) {
  if (a.row_index == nullptr) return r;
  const int64_t s = a.row_index[r];
  if (s >= 0 && s < a.x_rows) return s;
  set_status(a.status, GPTQ_ERR_INVALID_ARG);
  return -1;
}

// Largest finite magnitude of rows [r0, r1), columns [c0, c1), over the CTA.
template <bool BF16, bool NV>
__device__ __forceinline__ uint32_t region_max(const QuantArgs& a, int64_t r0, int64_t r1, int c0, int c1, uint32_t* s) {
  using S = Shape<BF16, NV>;
  const int across = (c1 - c0 + S::kBlock - 1) / S::kBlock;
  uint32_t m = 0;
  for (int64_t r = r0 + threadIdx.x / S::kCols; r < r1; r += S::kRowsAtOnce) {
    const int64_t src = source_row(a, r);
    if (src < 0) continue;
#pragma unroll 4
    for (int b = threadIdx.x % S::kCols; b < across; b += S::kCols) {
      uint32_t w[S::kWords];
      load_block<BF16, NV>(a, src, c0 + b * S::kBlock, w);
      m = max(m, finite_max<BF16>(w));
    }
  }
  return cta_max(m, s);
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

__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t k = c & 7;
  const float v = k < 2 ? 0.5f * k : __uint_as_float(((k >> 1) + 126) << 23 | (k & 1) << 22);
  return c & 8 ? -v : v;
}

// E4M3 byte nearest to amax / (6 t), decided on amax against the exact product
// of the border between two neighbours (5 bits) and 6 t (26 bits).
__device__ __noinline__ uint32_t exact_scale(float amax, float t, uint32_t lo, uint32_t hi) {
  for (uint32_t b = lo; b < hi; ++b) {
    const double border = 0.5 * (double(e4m3_value(b)) + double(e4m3_value(b + 1))) * (6.0 * double(t));
    if (amax < border || (amax == border && b % 2 == 0)) return b;
  }
  return hi;
}

// E2M1 code nearest to x / (s t), on the exact borders.
__device__ __noinline__ uint32_t exact_code(float x, float s, float t) {
  const double u = double(s) * double(t), a = fabs(double(x));
  uint32_t k = 0;
  while (k < 7) {
    const double border = 0.5 * (double(e2m1_value(k)) + double(e2m1_value(k + 1))) * u;
    if (a < border || (a == border && k % 2 == 0)) break;
    ++k;
  }
  return k | (__float_as_uint(x) >> 31) << 3;
}

struct Unit {  // what a CTA keeps of its group's tensor scale
  float t, c_lo, c_hi;      // c_lo <= 1 / (6 t) <= c_hi
  const float2* recip;      // shared: [scale byte] -> (r_lo, r_hi) around 1 / (s t)
};

// One block: codes, scale byte and s (NaN for a block with a value that is not
// finite: it must not pass for a number, and its codes are zero).
template <bool BF16, bool NV>
__device__ __forceinline__ void quantize_block(const uint32_t (&w)[Shape<BF16, NV>::kWords], const Unit& u,
                                               uint32_t (&codes)[Shape<BF16, NV>::kBlock / 8], uint32_t& byte, float& s) {
  using S = Shape<BF16, NV>;
  const uint32_t m = block_max<BF16>(w);
  if (m >= 0x7f800000u) {
    byte = NV ? 0x7f : 0xff;
    s = __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int i = 0; i < S::kBlock / 8; ++i) codes[i] = 0;
    return;
  }
  if (!NV) {
    const int lg = m >= 0x00800000u ? int(m >> 23) - 127 : m ? -118 - __clz(m) : -127;
    const int e = max(lg - 2, -127);
    byte = e + 127;
    s = e > -127 ? __uint_as_float(uint32_t(e + 127) << 23) : __uint_as_float(0x00400000u);
    const float inv = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < S::kBlock / 8; ++i) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = value<BF16>(w, 8 * i + j) * inv;
      codes[i] = to_e2m1(v);
    }
    return;
  }
  const float amax = __uint_as_float(m);
  const uint32_t two = to_e4m3x2(__fmul_rd(amax, u.c_lo), __fmul_ru(amax, u.c_hi));
  byte = two & 0xff;
  if (byte != two >> 8) byte = exact_scale(amax, u.t, byte, two >> 8);
  s = e4m3_value(byte);
  const float2 r = u.recip[byte];
  if (byte == 0) {
#pragma unroll
    for (int i = 0; i < S::kBlock / 8; ++i) codes[i] = 0;
    return;
  }
  uint32_t differ[S::kBlock / 8], any = 0;
#pragma unroll
  for (int i = 0; i < S::kBlock / 8; ++i) {
    float lo[8], hi[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      lo[j] = value<BF16>(w, 8 * i + j) * r.x;
      hi[j] = value<BF16>(w, 8 * i + j) * r.y;
    }
    codes[i] = to_e2m1(lo);
    differ[i] = codes[i] ^ to_e2m1(hi);
    if (!(r.y < FLT_MAX)) differ[i] = 0xffffffffu;  // 1 / (s t) is beyond a float
    any |= differ[i];
  }
  if (any != 0) {
#pragma unroll
    for (int i = 0; i < S::kBlock; ++i) {
      const int at = 4 * (i % 8);
      if (differ[i / 8] >> at & 15) codes[i / 8] = (codes[i / 8] & ~(15u << at)) | exact_code(value<BF16>(w, i), s, u.t) << at;
    }
  }
}

// The group of band `band` and its rows there; false past the last band.
struct Band {
  int g;
  int64_t r0;
  int rows;
  int64_t first, bands;    // the group's first band, and how many it has
  int64_t g0, g1;          // the group's rows
};

__device__ __forceinline__ bool find_band(const QuantArgs& a, const GroupTable& t, int64_t band, Band& b) {
  if (a.offsets != nullptr) {
    if (band >= t.band[a.groups]) return false;
    b.g = find_group(t.band, a.groups, static_cast<int>(band));
    b.first = t.band[b.g];
    b.bands = t.band[b.g + 1] - b.first;
    b.g0 = t.off[b.g];
    b.g1 = t.off[b.g + 1];
  } else {
    b.bands = (a.group_rows + kFp4Band - 1) / kFp4Band;
    if (b.bands == 0) return false;
    const int64_t g = band / b.bands;
    if (g >= a.groups) return false;
    b.g = static_cast<int>(g);
    b.first = g * b.bands;
    b.g0 = g * a.group_rows;
    b.g1 = b.g0 + a.group_rows;
  }
  b.r0 = b.g0 + (band - b.first) * kFp4Band;
  b.rows = static_cast<int>(min(static_cast<int64_t>(kFp4Band), b.g1 - b.r0));
  return true;
}

template <bool BF16, bool NV>
__global__ void __launch_bounds__(kThreads) fp4_amax_kernel(QuantArgs a) {
  __shared__ int tab[3][kFp4MaxGroups + 1];
  __shared__ uint32_t red[32];
  const GroupTable t{tab[0], tab[1], tab[2]};
  pdl_trigger();
  pdl_wait();
  if (a.offsets != nullptr && !build_groups(t, a.offsets, a.groups, a.rows, kFp4Band)) return;
  const int64_t band = blockIdx.x / a.splits;
  const int part = blockIdx.x % a.splits;
  Band b;
  if (!find_band(a, t, band, b)) return;
  const int chunks = (a.n + kChunk - 1) / kChunk;
  const int c0 = static_cast<int>(int64_t(chunks) * part / a.splits) * kChunk;
  const int c1 = min(a.n, static_cast<int>(int64_t(chunks) * (part + 1) / a.splits) * kChunk);
  const uint32_t m = region_max<BF16, NV>(a, b.r0, b.r0 + b.rows, c0, c1, red);
  if (threadIdx.x == 0) a.partial[blockIdx.x] = __uint_as_float(m);
}

template <bool BF16, bool NV>
__global__ void __launch_bounds__(kThreads) fp4_quantize_kernel(QuantArgs a) {
  using S = Shape<BF16, NV>;
  __shared__ int tab[3][kFp4MaxGroups + 1];
  __shared__ uint32_t red[32];
  __shared__ float2 recip[NV ? 128 : 1];
  __shared__ __align__(16) uint8_t sc[kFp4Band * (kChunk / S::kBlock)];
  const GroupTable t{tab[0], tab[1], tab[2]};
  pdl_trigger();
  pdl_wait();
  if (a.offsets != nullptr && !build_groups(t, a.offsets, a.groups, a.rows, kFp4Band)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, GPTQ_ERR_INVALID_ARG);
    return;
  }
  const int chunks = (a.n + kChunk - 1) / kChunk;
  const int64_t band = blockIdx.x / chunks;
  const int chunk = blockIdx.x % chunks;
  if (NV && !a.given && blockIdx.x == 0) {  // groups without rows have no CTA of their own
    for (int g = threadIdx.x; g < a.groups; g += kThreads)
      if (a.offsets != nullptr ? t.off[g] == t.off[g + 1] : a.group_rows == 0) a.tensor_scale[g] = FLT_MIN;
  }
  Band b;
  if (!find_band(a, t, band, b)) return;

  Unit u{1.0f, 0.0f, 0.0f, recip};
  if (NV) {
    if (a.given) {
      u.t = a.tensor_scale[b.g];
    } else {
      uint32_t m = 0;
      if (a.partial != nullptr) {
        const float* p = a.partial + b.first * a.splits;
        for (int64_t i = threadIdx.x; i < b.bands * a.splits; i += kThreads) m = max(m, __float_as_uint(p[i]));
        m = cta_max(m, red);
      } else {
        m = region_max<BF16, NV>(a, b.g0, b.g1, 0, a.n, red);
      }
      u.t = fmaxf(__fdiv_rn(__uint_as_float(m), 2688.0f), FLT_MIN);
      if (band == b.first && chunk == 0 && threadIdx.x == 0) a.tensor_scale[b.g] = u.t;
    }
    const double c = 1.0 / (6.0 * double(u.t));
    u.c_lo = __double2float_rd(c * (1.0 - 0x1p-50));
    u.c_hi = __double2float_ru(c * (1.0 + 0x1p-50));
    if (threadIdx.x < 127) {
      // one float further out than the nearest ones: the products x r_lo and
      // x r_hi are rounded themselves
      const double r = threadIdx.x > 0 ? 1.0 / (double(e4m3_value(threadIdx.x)) * double(u.t)) : 0.0;
      recip[threadIdx.x] = make_float2(nextafterf(__double2float_rd(r), 0.0f), nextafterf(__double2float_ru(r), INFINITY));
    }
  }
  for (int i = threadIdx.x; i < int(sizeof(sc)) / 4; i += kThreads) reinterpret_cast<uint32_t*>(sc)[i] = 0;
  __syncthreads();

  const int cb = threadIdx.x % S::kCols;
  const int col = chunk * kChunk + cb * S::kBlock;
  const int64_t pitch = fp4_pitch(a.n);
  if (col / 2 < pitch) {
    for (int it = 0; it < S::kIters; ++it) {
      const int r = it * S::kRowsAtOnce + threadIdx.x / S::kCols;
      if (r >= b.rows) break;
      const int64_t row = b.r0 + r;
      const int64_t src = source_row(a, row);
      uint32_t w[S::kWords];
      if (src >= 0 && col < a.n) {
        load_block<BF16, NV>(a, src, col, w);
      } else {
#pragma unroll
        for (int i = 0; i < S::kWords; ++i) w[i] = 0;
      }
      uint32_t codes[S::kBlock / 8], byte;
      float s;
      quantize_block<BF16, NV>(w, u, codes, byte, s);
      uint8_t* dst = a.packed + row * pitch + col / 2;
      if (NV)
        *reinterpret_cast<uint2*>(dst) = make_uint2(codes[0], codes[1]);
      else
        *reinterpret_cast<uint4*>(dst) = make_uint4(codes[0], codes[1], codes[S::kBlock / 8 - 2], codes[S::kBlock / 8 - 1]);
      if (col < a.n) sc[cb / 4 * kFp4TileBytes + r % 32 * 16 + r / 32 * 4 + cb % 4] = static_cast<uint8_t>(byte);
      if (a.deq != nullptr && col < a.n) {
        float* d = a.deq + row * a.n + col;
        const bool vec = a.n % 8 == 0 && col + S::kBlock <= a.n && reinterpret_cast<uintptr_t>(a.deq) % 32 == 0;
#pragma unroll
        for (int i = 0; i < S::kBlock / 8; ++i) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(e2m1_value(codes[i] >> 4 * j & 15) * s, u.t);
          if (vec) {
            store32(d + 8 * i, v);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (col + 8 * i + j < a.n) d[8 * i + j] = v[j];
          }
        }
      }
    }
  }
  __syncthreads();
  const int quads = fp4_quads(a.n, NV);
  const int q0 = chunk * (S::kCols / 4);
  const int bytes = min(S::kCols / 4, quads - q0) * kFp4TileBytes;
  uint8_t* out = a.scales + (band * quads + q0) * kFp4TileBytes;
  for (int i = threadIdx.x * 16; i < bytes; i += kThreads * 16)
    *reinterpret_cast<uint4*>(out + i) = *reinterpret_cast<const uint4*>(sc + i);
}

// Splits of a band's columns in the pass that takes the maxima: enough CTAs
// for the chip when there are few bands.
int amax_splits(int64_t bands, int n, int sms) {
  const int64_t chunks = ceil_div(n, kChunk);
  return static_cast<int>(std::min<int64_t>(chunks, std::max<int64_t>(1, ceil_div(4 * sms, bands))));
}

// Up to here every CTA reads its group's values itself instead of waiting for
// another kernel's maxima.
constexpr int64_t kSelfValues = 16384;

template <bool BF16, bool NV>
gptq_status launch_quantize(QuantArgs& a, int64_t bands, const DeviceInfo* info, cudaStream_t st) {
  const int64_t chunks = ceil_div(a.n, kChunk);
  if (a.partial != nullptr) {
    if (launch_pdl(fp4_amax_kernel<BF16, NV>, static_cast<unsigned>(bands * a.splits), kThreads, 0, st, a) != cudaSuccess)
      return GPTQ_ERR_CUDA;
  }
  if (launch_pdl(fp4_quantize_kernel<BF16, NV>, static_cast<unsigned>(bands * chunks), kThreads, 0, st, a) != cudaSuccess)
    return GPTQ_ERR_CUDA;
  return launch_status();
}

}  // namespace

size_t fp4_quantize_workspace_size(int64_t rows, int n, bool nv, int groups, bool ragged) {
  if (!nv || rows * n <= kSelfValues) return 0;
  const DeviceInfo* info = device_info();
  if (info == nullptr) return 0;
  const int64_t bands = fp4_bands(rows, groups, ragged);
  return static_cast<size_t>(bands * amax_splits(bands, n, info->sm_count)) * sizeof(float);
}

gptq_status fp4_quantize(const void* X, int x_bf16, int64_t x_rows, int n, int64_t ldx, const int32_t* row_index,
                         int64_t rows, const int32_t* offsets, int groups, bool nv, int given, float* tensor_scale,
                         uint8_t* packed, uint8_t* scales, float* deq, void* ws, cudaStream_t st) {
  const DeviceInfo* info = device_info();
  if (info == nullptr) return GPTQ_ERR_CUDA;
  const int64_t bands = std::max<int64_t>(1, fp4_bands(rows, groups, offsets != nullptr));
  QuantArgs a;
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
  a.packed = packed;
  a.scales = scales;
  a.deq = deq;
  a.given = given;
  a.splits = amax_splits(bands, n, info->sm_count);
  a.partial = nv && !given && rows * n > kSelfValues ? static_cast<float*>(ws) : nullptr;
  const uintptr_t at = reinterpret_cast<uintptr_t>(X) | static_cast<uintptr_t>(ldx * (x_bf16 ? 2 : 4));
  a.align = at % 32 == 0 ? 32 : at % 16 == 0 ? 16 : 0;
  a.status = info->status;
  if (nv)
    return x_bf16 ? launch_quantize<true, true>(a, bands, info, st) : launch_quantize<false, true>(a, bands, info, st);
  return x_bf16 ? launch_quantize<true, false>(a, bands, info, st) : launch_quantize<false, false>(a, bands, info, st);
}

}  // namespace gptq
