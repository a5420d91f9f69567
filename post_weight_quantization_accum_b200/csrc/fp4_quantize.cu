// Quantisation to 4-bit floating point (mxfp4, nvfp4).
//
//   mxfp4  blocks of 32: s = 2^(floor(log2 amax) - 2), clamped to 2^[-127, 127]
//   nvfp4  blocks of 16: t = max(RN(amax of the group / 2688), 2^-126),
//          s = E4M3 nearest to amax / (6 t), at most 448
//   code = E2M1 nearest to x / (s t), at most 6, ties to the even code
//
// The quotients are exact: which code is nearest is decided on the real
// numbers, not on rounded ones.  With mxfp4 dividing by s only moves the
// exponent.  With nvfp4 the quotient is bracketed: x r_lo < x / (s t) < x r_hi
// with r_lo and r_hi 2^-20 of it below and above 1 / (s t).  Where both ends
// convert to the same code the code is certain; where they do not (ties, above
// all: 3% of the blocks of bf16 values whose t was made from a bf16 maximum)
// the exact product b s t of the rounding border b, a float and its exact
// rest, is compared with x.  The scale is decided in the same way.
//
// Bound by HBM: per value 2 (bf16) or 4 (fp32) bytes in, 1/2 + 1/B out, and 4
// with the dequantised values.  A CTA takes a band of 128 rows x 256 columns
// (32 rows of it where there are few), a lane 32 bytes of a row at a time, so
// that a warp's loads are whole lines, with the next rows' loads in flight;
// the band's scale tiles go out whole from shared memory.  The tensor scales
// of nvfp4 take a pass of their own over X, whose end the second pass, which
// runs backwards, still finds in L2; a small X is read twice by the one
// kernel.  Measured with the values (B200): mxfp4 of fp32 11008 x 4096 63 us =
// 6.1 TB/s, 0.93 of the copy rate; nvfp4 of bf16 8192 x 4096 49 us = 4.5 TB/s
// on the bytes of one pass, 15 us of it the maxima (without the values 36 us,
// and 22 with a given tensor scale).  The second pass issues 305 instructions
// for a warp's 512 values, 256 without writing them: 55% and 71% of the cycles
// in which an SM has work.  Besides, with the values it waits for X, without
// them for the arithmetic pipes, and its 1024 CTAs on 592 places (1.7 waves)
// leave the SMs without work for 15 to 18% of the time.
#include <algorithm>

#include "fp4_quant.cuh"

namespace gptq {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 256;  // columns of a CTA's tile

// A lane's place in a CTA's tile.
template <bool BF16, bool NV>
struct Shape : Fp4Lane<BF16, NV> {
  static constexpr int kAcross = kChunk / Fp4Lane<BF16, NV>::kLane;  // lanes across the tile
  static constexpr int kRowsAtOnce = kThreads / kAcross;
  // rows loaded ahead of the one in work (8192 x 4096 of bf16 to nvfp4, second
  // pass: 39 us with 1, 46 with 2, which needs more registers)
  static constexpr int kAhead = NV ? 1 : 2;
};

// (the first to leave L2: what is read again is X)
__device__ __forceinline__ void store32(void* p, const float* v) {
  asm volatile("st.global.L1::no_allocate.L2::evict_first.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// What eight codes stand for.
__device__ __forceinline__ void from_e2m1(uint32_t codes, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint32_t cta_max(uint32_t m, uint32_t* s) {
  m = __reduce_max_sync(0xffffffffu, m);
  if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = m;
  __syncthreads();
  m = __reduce_max_sync(0xffffffffu, threadIdx.x % 32 < kThreads / 32 ? s[threadIdx.x % 32] : 0u);
  __syncthreads();
  return m;
}

// The source rows of a band, once for the whole CTA (a gather's indices are
// then not waited for row by row).
__device__ __forceinline__ void band_rows(const QuantArgs& a, int64_t r0, int rows, int* src) {
  if (threadIdx.x < rows) src[threadIdx.x] = source_row(a, r0 + threadIdx.x);
  __syncthreads();
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

// A thread's part of the largest magnitude of chunk c of a band's rows on any
// place: the whole 16-byte pieces of a row that start in the chunk, and the
// row's two ends.  (Out of line: other calls do not fetch its code.)
template <bool BF16>
__device__ __noinline__ uint32_t chunk_max(const QuantArgs& a, const int* src, int rows, int c) {
  constexpr int kSize = BF16 ? 2 : 4, kBytes = kChunk * kSize;
  const char* X = static_cast<const char*>(a.X);
  const int end = a.n * kSize;
  const bool last = end <= (c + 1) * kBytes;
  return runs_max<BF16, kBytes / 16>(threadIdx.x, kThreads, rows, 0, c == 0 || last, [&](int r, const char*& lo, const char*& hi) {
    const int row = src[r];
    if (row < 0) return;
    const char* x = X + row * a.ldx * kSize;
    const int shift = -reinterpret_cast<uintptr_t>(x) & 15, whole = end - ((end - shift) & 15);  // of the last piece's end
    lo = x + (c == 0 ? 0 : min(c * kBytes + shift, whole));
    hi = x + (last ? end : min((c + 1) * kBytes + shift, whole));
  });
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) fp4_amax_kernel(const __grid_constant__ QuantArgs a) {
  __shared__ int tab[3][kFp4MaxGroups + 1];
  __shared__ uint32_t red[32];
  __shared__ int src[kFp4Band];
  const GroupTable t{tab[0], tab[1], tab[2]};
  pdl_wait();
  pdl_trigger();  // (after the wait: what starts now may read all that was written before this kernel)
  if (a.offsets != nullptr && !build_groups(t, a.offsets, a.groups, a.rows, kFp4Band)) return;
  const int64_t band = blockIdx.x / a.splits;
  const int part = blockIdx.x % a.splits;
  Band b;
  if (!find_band(a, t, band, b)) return;
  const int chunks = (a.n + kChunk - 1) / kChunk;
  // this part's columns, a chunk after the other, each down the band's rows
  using S = Shape<BF16, true>;
  band_rows(a, b.r0, b.rows, src);
  const int c0 = static_cast<int>(int64_t(chunks) * part / a.splits), c1 = static_cast<int>(int64_t(chunks) * (part + 1) / a.splits);
  const char* X = static_cast<const char*>(a.X);
  constexpr int kSize = BF16 ? 2 : 4;
  uint32_t m = 0;
  for (int c = c0; c < c1; ++c) {
    uint32_t t;
    if (a.vec == 0) {
      t = chunk_max<BF16>(a, src, b.rows, c);
    } else {
      const int col = c * kChunk + threadIdx.x % S::kAcross * S::kLane, r = threadIdx.x / S::kAcross;
      auto at = [&](int r, int& left) -> const char* {
        const int row = src[r];
        left = a.n - col;
        return row < 0 || left <= 0 ? nullptr : X + (row * a.ldx + col) * kSize;
      };
      t = a.vec == 2 && (c + 1) * kChunk <= a.n ? thread_max<BF16, 2, 4>(a, r, S::kRowsAtOnce, b.rows, at)
                                                : thread_max<BF16, 0, 4>(a, r, S::kRowsAtOnce, b.rows, at);
    }
    m = max(m, t);
  }
  m = cta_max(m, red);
  if (threadIdx.x == 0) a.partial[blockIdx.x] = __uint_as_float(m);
}

// Whether the rows of the dequantised values start on 32 bytes.
__device__ __forceinline__ bool wide_values(const QuantArgs& a) {
  return a.n % 8 == 0 && reinterpret_cast<uintptr_t>(a.deq) % 32 == 0;
}

// A lane's values down the band's rows.  VEC: whole loads (load_lane), and
// 32-byte stores of the values that they stand for.  (Rows of 2056 bf16 start
// on 16 bytes: 24.6 us with VEC 1, 25.4 with the loads that look at each place.)
template <bool BF16, bool NV, int VEC>
__device__ __forceinline__ void quantize_rows(const QuantArgs& a, const Band& b, const Unit& u, const int* src, int col,
                                              int64_t pitch, uint8_t* sc, float* stage) {
  using S = Shape<BF16, NV>;
  constexpr int kSize = BF16 ? 2 : 4;
  const char* X = static_cast<const char*>(a.X);
  const int left = a.n - col, chunk0 = col - threadIdx.x % S::kAcross * S::kLane;
  // values go out in 32-byte stores, or, where their rows do not start on 32
  // bytes, through shared memory (512 floats a warp) as whole lines
  const bool wide = VEC != 0 || wide_values(a);
  constexpr int kRowsWarp = 32 / S::kAcross;  // rows of a warp
  float* mine = stage + threadIdx.x / 32 * 512;
  const int cb = threadIdx.x % S::kAcross / S::kLanes;  // block of the chunk
  const bool first = threadIdx.x % S::kLanes == 0 && left > 0;  // the lane that writes the block's scale
  uint8_t* sc_col = sc + cb / 4 * kFp4TileBytes + cb % 4;
  auto at = [&](int r) -> const char* {
    const int row = r < b.rows ? src[r] : -1;
    return row < 0 || left <= 0 ? nullptr : X + (row * a.ldx + col) * kSize;
  };
  auto fetch = [&](const char* p, uint32_t (&w)[8]) {
    if (p != nullptr) {
      load_lane<BF16, VEC>(p, left, col, w);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 0;
    }
  };
  uint32_t w[S::kAhead + 1][8];
  const char* p[S::kAhead + 1];
  int r = threadIdx.x / S::kAcross;
#pragma unroll
  for (int v = 0; v < S::kAhead; ++v) {
    p[v] = at(r + v * S::kRowsAtOnce);
    fetch(p[v], w[v]);
  }
  uint8_t* dst = a.packed + (b.r0 + r) * pitch + col / 2;
  float* deq = a.deq + (b.r0 + r) * a.n + col;
#pragma unroll 2
  for (int r0 = 0; r0 < b.rows; r0 += S::kRowsAtOnce, r += S::kRowsAtOnce) {  // (as often in every lane)
    p[S::kAhead] = at(r + S::kAhead * S::kRowsAtOnce);
    fetch(p[S::kAhead], w[S::kAhead]);
    uint32_t codes[S::kLane / 8], byte;
    float s;
    quantize_lane<BF16, NV>(w[0], p[0], left, u, codes, byte, s);
    if (r < b.rows) {
      if (col / 2 < pitch) {
        if (BF16)
          *reinterpret_cast<uint2*>(dst) = make_uint2(codes[0], codes[S::kLane / 8 - 1]);
        else
          *reinterpret_cast<uint32_t*>(dst) = codes[0];
      }
      if (first) sc_col[r % 32 * 16 + r / 32 * 4] = static_cast<uint8_t>(byte);
    }
    if (a.deq != nullptr) {
#pragma unroll
      for (int i = 0; i < S::kLane / 8; ++i) {
        float f[8];
        from_e2m1(codes[i], f);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          mul2(f[j], f[j + 1], f[j], f[j + 1], s);
          if (NV) mul2(f[j], f[j + 1], f[j], f[j + 1], u.t);
        }
        if (!wide) {
          float4* m = reinterpret_cast<float4*>(mine + threadIdx.x % 32 * S::kLane + 8 * i);
          m[0] = make_float4(f[0], f[1], f[2], f[3]);
          m[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else if (r < b.rows && 8 * i < left) {
          store32(deq + 8 * i, f);
        }
      }
      if (!wide) {
        __syncwarp();
        const int lane = threadIdx.x % 32, row0 = r - threadIdx.x % 32 / S::kAcross;
#pragma unroll
        for (int q = 0; q < kRowsWarp; ++q) {
          float* out = a.deq + (b.r0 + row0 + q) * a.n + chunk0 + lane;
#pragma unroll
          for (int i = 0; i < kChunk / 32; ++i)
            if (row0 + q < b.rows && chunk0 + 32 * i + lane < a.n) out[32 * i] = mine[q * kChunk + 32 * i + lane];
        }
        __syncwarp();
      }
    }
    dst += S::kRowsAtOnce * pitch;
    deq += static_cast<int64_t>(S::kRowsAtOnce) * a.n;
#pragma unroll
    for (int v = 0; v < S::kAhead; ++v) {
      p[v] = p[v + 1];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[v][i] = w[v + 1][i];
    }
  }
}

// A thread's part of the largest magnitude of `count` rows from row g0 on.  (Out
// of line: kernels that do not take it otherwise paid 1 to 2 us for its code.)
template <bool BF16>
__device__ __noinline__ uint32_t group_max(const QuantArgs& a, int64_t g0, int count) {
  constexpr int kSize = BF16 ? 2 : 4;
  const char* X = static_cast<const char*>(a.X);
  const int bytes = a.n * kSize;
  if (a.row_index == nullptr && a.ldx == a.n) {  // one run
    const char* first = X + g0 * bytes;
    const bool ends = (reinterpret_cast<uintptr_t>(first) | (count * bytes)) % 16 != 0;
    return runs_max<BF16, 0>(threadIdx.x, kThreads, 1, count * bytes / 16, ends, [&](int, const char*& lo, const char*& hi) {
      lo = first;
      hi = lo + count * bytes;
    });
  }
  return runs_max<BF16, 0>(threadIdx.x, kThreads, count, max(bytes / 16, 1), a.vec == 0 || bytes % 16 != 0,
                           [&](int r, const char*& lo, const char*& hi) {
                             const int row = source_row(a, g0 + r);
                             if (row < 0) return;
                             lo = X + row * a.ldx * kSize;
                             hi = lo + bytes;
                           });
}

template <bool BF16, bool NV>
__global__ void __launch_bounds__(kThreads, 4) fp4_quantize_kernel(const __grid_constant__ QuantArgs a) {
  using S = Shape<BF16, NV>;
  __shared__ int tab[3][kFp4MaxGroups + 1];
  __shared__ uint32_t red[32];
  __shared__ int src[kFp4Band];
  __shared__ __align__(16) float stage[kThreads * 16];
  __shared__ __align__(16) uint8_t sc[kFp4Band * (kChunk / S::kBlock)];
  const GroupTable t{tab[0], tab[1], tab[2]};
  auto start = [] {
    pdl_wait();
    pdl_trigger();  // (after the wait: what starts now may read all that was written before this kernel)
  };
  // After a pass for the maxima, which let this kernel start when all before it
  // was done, only the maxima are waited for (8192 x 4096: 51 -> 49 us; 6000
  // gathered rows of 2056 in 24 groups: 26.1 -> 25.0).
  const bool after = NV && a.partial != nullptr;
  if (!after) start();
  if (a.offsets != nullptr && !build_groups(t, a.offsets, a.groups, a.rows, kFp4Band)) {
    if (after) start();
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, GPTQ_ERR_INVALID_ARG);
    return;
  }
  const int chunks = (a.n + kChunk - 1) / kChunk;
  // (after a pass for the maxima: from its end, whose values are still in L2)
  const unsigned at = after ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
  const int64_t band = at / chunks / a.strips;
  const int strip = at / chunks % a.strips, chunk = at % chunks;
  if (NV && !a.given && blockIdx.x == 0) {  // groups without rows have no CTA of their own
    if (after) pdl_wait();
    for (int g = threadIdx.x; g < a.groups; g += kThreads)
      if (a.offsets != nullptr ? t.off[g] == t.off[g + 1] : a.group_rows == 0) a.tensor_scale[g] = FLT_MIN;
  }
  Band b;
  if (!find_band(a, t, band, b)) {
    if (after) start();
    return;
  }
  const int height = kFp4Band / a.strips;
  b.r0 += strip * height;
  b.rows = max(0, min(height, b.rows - strip * height));
  if (b.rows < height || (chunk + 1) * kChunk > a.n) {  // bytes that have no row or block are zero
    for (int i = threadIdx.x; i < int(sizeof(sc)) / 4; i += kThreads) reinterpret_cast<uint32_t*>(sc)[i] = 0;
  }
  band_rows(a, b.r0, b.rows, src);
  if (after) start();

  Unit u{1.0f, 1.0f, 1.0f, true};
  if (NV) {
    float tensor;
    if (a.given) {
      tensor = a.tensor_scale[b.g];
    } else {
      uint32_t m = 0;
      if (a.partial != nullptr) {
        const float* p = a.partial + b.first * a.splits;
        for (int64_t i = threadIdx.x; i < b.bands * a.splits; i += kThreads) m = max(m, __float_as_uint(p[i]));
        m = cta_max(m, red);
      } else {
        m = group_max<BF16>(a, b.g0, static_cast<int>(b.g1 - b.g0));
        m = cta_max(m, red);
      }
      tensor = fmaxf(__fdiv_rn(__uint_as_float(m), 2688.0f), FLT_MIN);
      if (band == b.first && chunk == 0 && strip == 0 && threadIdx.x == 0) a.tensor_scale[b.g] = tensor;
    }
    u = unit_of(tensor);
  }

  const int col = chunk * kChunk + threadIdx.x % S::kAcross * S::kLane;
  const int64_t pitch = fp4_pitch(a.n);
  const int vec = (chunk + 1) * kChunk <= a.n && (a.deq == nullptr || wide_values(a)) ? a.vec : 0;
  if (vec == 2)
    quantize_rows<BF16, NV, 2>(a, b, u, src, col, pitch, sc, stage);
  else if (vec == 1)
    quantize_rows<BF16, NV, 1>(a, b, u, src, col, pitch, sc, stage);
  else
    quantize_rows<BF16, NV, 0>(a, b, u, src, col, pitch, sc, stage);
  __syncthreads();
  const int quads = fp4_quads(a.n, NV);
  constexpr int kQuads = kChunk / (4 * S::kBlock);  // scale tiles across the chunk
  const int q0 = chunk * kQuads;
  const int bytes = min(kQuads, quads - q0) * kFp4TileBytes;
  uint8_t* out = a.scales + (band * quads + q0) * kFp4TileBytes;
  if (a.strips == 1) {
    for (int i = threadIdx.x * 16; i < bytes; i += kThreads * 16)
      *reinterpret_cast<uint4*>(out + i) = *reinterpret_cast<const uint4*>(sc + i);
  } else {  // rows 32 strip .. 32 strip + 31 are the strip-th word of each 16 bytes, and stand at the first in `sc`
    for (int i = threadIdx.x * 16; i < bytes; i += kThreads * 16)
      *reinterpret_cast<uint32_t*>(out + i + 4 * strip) = *reinterpret_cast<const uint32_t*>(sc + i);
  }
}

// Parts of a band's columns in the pass that takes the maxima: a chunk each, or
// several, down to one part a band, where that would leave over 2048 maxima.
// Every CTA of the second pass reads all of its group's: 8 KB up to 2048 bands
// (262,144 rows), 4 bytes a band above (2^20 x 4096: 32 KB in each of 131,072
// CTAs, half as much as bf16 values of X, though out of L2).
int amax_splits(int64_t bands, int n) {
  const int64_t chunks = ceil_div(n, kChunk);
  return static_cast<int>(ceil_div(chunks, std::max<int64_t>(1, ceil_div(bands * chunks, 2048))));
}

template <bool BF16, bool NV>
gptq_status launch_quantize(QuantArgs& a, int64_t bands, const DeviceInfo* info, cudaStream_t st) {
  const int64_t chunks = ceil_div(a.n, kChunk);
  // few bands: a CTA takes 32 rows of one, so that more SMs have work (a layer
  // on 128 tokens, nvfp4, 4096 -> 11008: 21.2 us with whole bands, 17.2 with 32)
  a.strips = bands * chunks <= info->sm_count && a.rows > 32 ? 4 : 1;
  if constexpr (NV) {
    if (a.partial != nullptr &&
        launch_pdl(fp4_amax_kernel<BF16>, static_cast<unsigned>(bands * a.splits), kThreads, 0, st, a) != cudaSuccess)
      return GPTQ_ERR_CUDA;
  }
  if (launch_pdl(fp4_quantize_kernel<BF16, NV>, static_cast<unsigned>(bands * a.strips * chunks), kThreads, 0, st, a) != cudaSuccess)
    return GPTQ_ERR_CUDA;
  return launch_status();
}

}  // namespace

size_t fp4_quantize_workspace_size(int64_t rows, int n, bool nv, int groups, bool ragged) {
  if (!nv || fp4_self_max(rows, n, groups, ragged)) return 0;
  const int64_t bands = fp4_bands(rows, groups, ragged);
  return static_cast<size_t>(bands * amax_splits(bands, n)) * sizeof(float);
}

gptq_status fp4_quantize(const void* X, int x_bf16, int64_t x_rows, int n, int64_t ldx, const int32_t* row_index,
                         int64_t rows, const int32_t* offsets, int groups, bool nv, int given, float* tensor_scale,
                         uint8_t* packed, uint8_t* scales, float* deq, void* ws, cudaStream_t st) {
  const DeviceInfo* info = device_info();
  if (info == nullptr) return GPTQ_ERR_CUDA;
  const int64_t bands = std::max<int64_t>(1, fp4_bands(rows, groups, offsets != nullptr));
  QuantArgs a = fp4_quant_args(X, x_bf16, x_rows, n, ldx, row_index, rows, offsets, groups, given, tensor_scale, info->status);
  a.packed = packed;
  a.scales = scales;
  a.deq = deq;
  a.splits = amax_splits(bands, n);
  a.partial = nv && !given && !fp4_self_max(rows, n, groups, offsets != nullptr) ? static_cast<float*>(ws) : nullptr;
  if (nv)
    return x_bf16 ? launch_quantize<true, true>(a, bands, info, st) : launch_quantize<false, true>(a, bands, info, st);
  return x_bf16 ? launch_quantize<true, false>(a, bands, info, st) : launch_quantize<false, false>(a, bands, info, st);
}

}  // namespace gptq
