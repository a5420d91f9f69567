// Sizes and shapes of the launches of the 4-bit products that need no GPU:
// plain C++, so that they can be checked on the host for every size.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "pair_left.h"

namespace gptq {

constexpr int kFp4Band = 128;        // rows of a scale tile
constexpr int kFp4TileBytes = 512;   // 128 rows x 4 blocks
constexpr int kFp4MaxGroups = 512;   // groups of an offsets array
// Up to here the CTAs of a product quantise its tokens themselves, each all of
// its part of K and, for the maximum, each all values.
constexpr int64_t kFp4RawValues = 16384;

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kRows = 128;    // weight rows of a CTA's tile
constexpr int kStageK = 256;  // columns of K a stage (128 bytes)
constexpr int kBoxRows = 32;  // token rows a TMA box
constexpr int kBoxBytes = kBoxRows * kStageK / 2;
constexpr int kABytes = kRows * kStageK / 2;
constexpr int kSfBytes = kStageK / 64 * kFp4TileBytes;  // scales of 128 rows of a stage (nvfp4; half of it with mxfp4)

// ---------------------------------------------------------------------------
// the kernel for few tokens
// ---------------------------------------------------------------------------

constexpr int kStreamMaxStages = 8;
constexpr int kStreamBarBytes = 384;
constexpr int kPushTokens = 16;      // up to here sums are sent (an MMA's least columns)
constexpr int kRawTokens = 16;       // of a RAW tile: one MMA's least columns
constexpr int kRawMaxStages = 8;     // of a RAW CTA's K range
constexpr int kRawStageBytes = kRawTokens * kStageK / 2 + kSfBytes;

struct StreamShape {
  int width;   // tokens of a tile: 16, 32, 64 or 128
  int stages;
  int splits;  // CTAs of a cluster
  int accs;    // accumulators: 2 where a CTA walks over tiles
  int raw_stages;  // RAW: most stages of a CTA's K range
};
inline GPTQ_HD int stream_stage_bytes(int width, bool raw) {
  return kABytes + (raw ? 0 : (width < kBoxRows ? kBoxRows : width) * (kStageK / 2) + kSfBytes) + kSfBytes;
}
inline GPTQ_HD int table_bytes(int groups) { return 3 * (groups + 1) * 4; }
// Shared memory in which a CTA of a split collects sums: for each of the
// `splits` sources the same number of rows of 128 floats (so up to splits - 1
// rows more than the tokens).  Up to 32 tokens it stands apart; more use the
// operand ring again, which is larger than 128 rows.
inline GPTQ_HD int stream_apart_bytes(int width, int splits) {
  const int bytes = splits * ((width + splits - 1) / splits) * kRows * 4;
  return splits > 1 && width <= 32 ? (bytes + 1023) / 1024 * 1024 : 0;  // (an operand may follow)
}
// Tensor memory of a CTA: accumulators and 32 scale columns a stage (at most
// 2 * 128 + 32 * 8).
inline GPTQ_HD uint32_t stream_tmem_cols(int width, int accs, int stages) {
  const int need = accs * width + 32 * stages;
  return need > 256 ? 512 : need > 128 ? 256 : 128;
}
constexpr size_t kStreamMaxSmem = 226 * 1024;
// A walking CTA has the SM to itself: what its ring may take.
constexpr int kWalkRingBytes = 200 * 1024;
// Shared memory of two CTAs that share an SM: half of its 228 KB, less 1 KB that
// the system keeps of each CTA's.
constexpr size_t kStreamTwoSmem = 228 * 1024 / 2 - 1024;

// Shared memory of a CTA: alignment, ring, sums, RAW tokens, barriers, groups.
inline size_t stream_smem(const StreamShape& s, bool raw, int groups) {
  return 1024 + static_cast<size_t>(s.stages) * stream_stage_bytes(s.width, raw) + stream_apart_bytes(s.width, s.splits) +
         (raw ? s.raw_stages * kRawStageBytes : 0) + kStreamBarBytes + table_bytes(groups);
}

// Tiles that a launch may have (each group's last one may be part full).
inline int64_t stream_tiles(const StreamShape& s, int64_t tokens, int groups, bool ragged, int64_t rows) {
  return (ragged ? tokens / s.width + std::min<int64_t>(groups, tokens) : div_up(tokens, s.width)) * div_up(rows, kRows);
}

// How few tokens are laid out.  Tiles are as wide as the tokens; groups, whose
// sizes the host does not know, take 64: they come here up to 32 tokens each on
// average, twice that fills a tile, and a group's second tile then starts at the
// third scale column of its band (a narrower one would start inside a column).
// Clusters are chosen for the stages of K that the busiest SM works off: two
// CTAs that walk over whole tiles and share an odd last one, or k CTAs a tile.
// (One token, n = 4096: 32 row tiles take 4 CTAs each; 48 tokens, 86 row tiles:
// 3 each, 12 stages instead of 16.)
inline StreamShape stream_shape(int64_t tokens, int groups, bool ragged, int64_t rows, int n, int sms) {
  StreamShape s;
  const int64_t each = ragged ? 64 : tokens;
  s.width = each <= 16 ? 16 : each <= 32 ? 32 : each <= 64 ? 64 : 128;
  s.raw_stages = 0;
  const int kstages = static_cast<int>(div_up(n, kStageK));
  const int64_t tiles = (ragged ? std::min<int64_t>(groups, tokens) : div_up(tokens, s.width)) * div_up(rows, kRows);
  const int64_t share = div_up(tiles, std::max(1, sms / 2));  // tiles of a walking pair
  int64_t best = kstages >= 2 ? share / 2 * kstages + share % 2 * ((kstages + 1) / 2) : div_up(tiles, sms);
  s.splits = 0;
  for (int k = 2; k <= 8 && k <= kstages && tiles * k <= 2 * sms; ++k) {  // (more would not run side by side)
    const int64_t cost = div_up(tiles * k, sms) * div_up(kstages, k);
    if (cost < best || (cost == best && s.splits == 0)) {
      best = cost;
      s.splits = k;
    }
  }
  s.accs = s.splits == 0 ? 2 : 1;
  s.stages = s.accs == 2 ? std::min(kStreamMaxStages, kWalkRingBytes / stream_stage_bytes(s.width, false))
                         : s.width <= 16 ? 4 : 3;  // (two CTAs an SM, with 32 rows of sums apart)
  if (s.splits == 0) s.splits = kstages >= 2 ? 2 : 1;
  return s;
}

// How the product quantises X itself, or false where X is quantised first: a
// few tokens whose values every CTA may read, and a K range that its shared
// memory holds.
inline bool raw_shape(int64_t tokens, int groups, bool ragged, int64_t rows, int n, int sms, StreamShape* s) {
  if (tokens > kRawTokens || tokens * n > kFp4RawValues) return false;
  *s = stream_shape(tokens, groups, ragged, rows, n, sms);  // (the splits, and so the sums, of the two calls)
  if (s->accs == 2) return false;  // (it walks)
  s->width = kRawTokens;
  s->stages = 4;
  s->raw_stages = static_cast<int>(div_up(div_up(n, kStageK), s->splits));
  // The cut counts on two CTAs an SM.  With 8 stages of tokens (or 7, and over
  // 300 groups) a ring of 4 leaves room for one, so a launch of more CTAs than
  // SMs takes 3 (one token in bf16, nvfp4, 4096 -> 14336: 11.5 us with 3, 17.1
  // with 4 in two rounds; 14336 -> 5120 21.6 and 27.8).
  if (stream_smem(*s, true, groups) > kStreamTwoSmem && stream_tiles(*s, tokens, groups, ragged, rows) * s->splits > sms) s->stages = 3;
  return s->raw_stages <= kRawMaxStages;
}

}  // namespace gptq
