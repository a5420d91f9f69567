// The 4-bit floating-point formats shared by the quantiser and the products.
//
// A matrix [rows, n] is held as
//   packed  E2M1 codes, two a byte (even column in the low half), each row
//           padded with zero codes to 32 columns: 16 * ceil(n / 32) bytes;
//   scales  one byte a block of columns, in tiles of 128 rows x 4 blocks: 512
//           bytes, the byte of row r and block b at
//           16 (r % 32) + 4 (r / 32 % 4) + b % 4, tiles of one 128-row band in
//           column order.  This is the order in which tensor memory wants the
//           scales of 128 rows (lane r % 32, column r / 32, byte b % 4), so a
//           tile goes there with one copy and no shuffling;
//   t       one fp32 scale a group of rows (nvfp4), or none (mxfp4).
// Groups of rows (experts) each start a new band of 128, so that a band's
// scales belong to one group wherever the group's rows begin.
#pragma once

#include "common.cuh"
#include "fp4_shape.h"

namespace gptq {

inline __host__ __device__ int fp4_block(bool nv) { return nv ? 16 : 32; }
inline __host__ __device__ int64_t fp4_pitch(int n) { return int64_t(16) * ((n + 31) / 32); }
// scale tiles along a row
inline __host__ __device__ int fp4_quads(int n, bool nv) { return (n + 4 * fp4_block(nv) - 1) / (4 * fp4_block(nv)); }

// Bands that `rows` rows in `groups` groups can take: each group's last band
// may be part full.  Exact for groups of one size (ragged == false).
inline int64_t fp4_bands(int64_t rows, int64_t groups, bool ragged) {
  if (!ragged) return groups * ceil_div(rows / groups, kFp4Band);
  return rows / kFp4Band + groups;
}

// What a CTA keeps of the groups: off[g] = first row, band[g] = first scale
// band, tile[g] = first tile of `width` rows; entry `groups` holds the ends.
// Built by the whole CTA; false (for every thread) when the offsets fall,
// leave [0, total] or are negative, in which case nothing may be read by them.
struct GroupTable {
  int* off;
  int* band;
  int* tile;
};

__device__ __forceinline__ bool build_groups(const GroupTable& t, const int32_t* __restrict__ offsets, int groups,
                                             int64_t total, int width) {
  __shared__ int bad_s;
  for (int i = threadIdx.x; i <= groups; i += blockDim.x) t.off[i] = offsets[i];
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    bool bad = t.off[0] < 0 || t.off[groups] > total;
    int carry_b = 0, carry_t = 0;
    for (int base = 0; base < groups; base += 32) {
      const int g = base + lane;
      const int64_t c64 = g < groups ? int64_t(t.off[g + 1]) - t.off[g] : 0;
      bad |= c64 < 0;
      const int c = c64 < 0 || c64 > total ? 0 : static_cast<int>(c64);
      int b = (c + kFp4Band - 1) / kFp4Band, w = (c + width - 1) / width;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int ub = __shfl_up_sync(0xffffffffu, b, d), uw = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) {
          b += ub;
          w += uw;
        }
      }
      if (g < groups) {
        t.band[g + 1] = carry_b + b;
        t.tile[g + 1] = carry_t + w;
      }
      carry_b += __shfl_sync(0xffffffffu, b, 31);
      carry_t += __shfl_sync(0xffffffffu, w, 31);
    }
    if (lane == 0) t.band[0] = t.tile[0] = 0;
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) bad_s = bad;
  }
  __syncthreads();
  return !bad_s;
}

// The group of entry `at` of a rising prefix p[0 .. groups] (p[0] = 0,
// at < p[groups]): the last g with p[g] <= at, so never an empty one.
__device__ __forceinline__ int find_group(const int* p, int groups, int at) {
  int lo = 0, hi = groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p[mid] <= at)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

}  // namespace gptq
