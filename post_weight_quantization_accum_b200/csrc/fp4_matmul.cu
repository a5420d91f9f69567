// Products of 4-bit floating-point matrices on the tensor cores, dense and
// grouped by expert:
//
//   y[i, r] = tw[g] tx[g] sum_c W[g, r, c] X[i, c],  i in group g's rows of X
//
// with both operands as E2M1 codes and block scales (fp4.cuh).  The block
// scales are multiplied in by the tensor cores (tcgen05.mma .block_scale), the
// sums are fp32, the tensor scales are multiplied in at the end.
//
// Roles are turned round against the usual: the M rows of an MMA are rows of W
// and its N columns are tokens, so that a single token is an MMA of N = 16 and
// every group's last tile only as wide as its tokens.  TMA brings 256 columns
// of K a stage (128 bytes a row, 128-byte swizzle) and the stage's scale
// tiles; tcgen05.cp takes those to tensor memory.
//
// Two kernels: few tokens a group (fp4_stream_kernel, bound by streaming W)
// and many (fp4_pair_kernel, bound by the tensor cores and the shared memory
// that feeds them).
#include <algorithm>
#include <atomic>

#include "fp4_quant.cuh"

namespace gptq {
namespace {

constexpr int kTokens = 256;  // tokens of a pair's tile at most
constexpr uint64_t kDrainNs = 2000000000ull;

struct MatmulArgs {
  const uint8_t* wscales;
  const uint8_t* xscales;
  const float* wt;  // tensor scales of each group; nullptr: 1
  const float* xt;
  const int32_t* offsets;
  int groups;
  int64_t rows;    // of W in each group
  int64_t tokens;
  int n;
  void* y;
  int64_t ldy;
  int early;  // the kernel before this one is the quantiser of X, which starts it
              // after its own wait: W and the offsets are there from the start
  int* status;
  uint64_t wait_ns;
};

// D (+)= A B^T with block scales: kind::mxf4nvf4 has a scale every 16 columns
// (E4M3), kind::mxf4 every 32 (2^e).  CTAS = 2: the pair form (the even CTA
// issues; each CTA holds half of A's rows and half of B's, and the scales of
// its own A rows and of all B rows).
#define GPTQ_FP4_MMA(GROUP, KIND)                                                                              \
  asm volatile(                                                                                                \
      "{\n\t.reg .pred p;\n\t"                                                                                \
      "setp.ne.b32 p, %6, 0;\n\t"                                                                              \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),        \
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                                  \
      : "memory")
template <bool NV, int CTAS>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
  if (NV && CTAS == 1)
    GPTQ_FP4_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
  else if (NV)
    GPTQ_FP4_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
  else if (CTAS == 1)
    GPTQ_FP4_MMA("1", "mxf4.block_scale.scale_vec::2X");
  else
    GPTQ_FP4_MMA("2", "mxf4.block_scale.scale_vec::2X");
}
#undef GPTQ_FP4_MMA

// Instruction descriptor of the block-scaled kinds: E2M1 operands along K,
// scale type (0 E4M3, 1 2^e), M = 128 a CTA, N tokens; `pair` picks the byte
// pair of the 32-bit scale cell (mxfp4 uses two bytes an MMA).
__device__ __forceinline__ uint32_t fp4_idesc(bool nv, uint32_t ctas, uint32_t n, uint32_t pair) {
  return (pair * 2) << 4 | 1u << 7 | 1u << 10 | (n >> 3) << 17 | (nv ? 0u : 1u) << 23 | ctas << 27 | (pair * 2) << 29;
}

// A scale tile (512 bytes of shared memory, 32 rows of 16 bytes) to four
// tensor-memory columns, the same for each quarter of the lanes (CTAS = 2: in
// both CTAs, each from its own shared memory).
template <int CTAS>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t smem) {
  const uint64_t desc = static_cast<uint64_t>((smem >> 4) & 0x3FFFu) | 8ull << 32 | 1ull << 46;  // 8 rows apart: 128 bytes
  if (CTAS == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Waits for a barrier's phase until the limit or until another role of the CTA
// has given up; the first to run out records the timeout.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile int* abort_flag, int* status) {
  const uint64_t t0 = global_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_ns() - t0 > limit_ns) {
      set_status(status, GPTQ_ERR_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
}

struct Tile {
  int g;
  int token;      // first token (row of X)
  int count;      // tokens of the tile
  int cols;       // MMA columns: count rounded up to 16
  int xband;      // first band of X's scales
  int xcol;       // tensor-memory column (32 tokens each) of the first token in that band
  int wtile;      // tile of W's rows in the group
};

// The two tensor scales of a group as factors of its sums: their product, or
// each in turn where the product would leave the normal numbers.
struct Scale {
  float k;
  float before;  // 1 where k is the product
};
__device__ __forceinline__ Scale make_scale(float tw, float tx) {
  const float k = tw * tx;
  if (k >= 1.17549435e-38f && k <= 3.40282347e38f) return {k, 1.0f};
  return {tx, tw};
}
__device__ __forceinline__ Scale tile_scale(const MatmulArgs& a, int g) {
  return a.wt == nullptr ? Scale{1.0f, 1.0f} : make_scale(a.wt[g], a.xt[g]);
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Four features of a token, of which `left` exist.
__device__ __forceinline__ void store_four(float* p, float4 v, Scale k, bool vec, int64_t left) {
  const float4 o = make_float4(v.x * k.before * k.k, v.y * k.before * k.k, v.z * k.before * k.k, v.w * k.before * k.k);
  if (vec) {
    *reinterpret_cast<float4*>(p) = o;
  } else {
    if (left > 0) p[0] = o.x;
    if (left > 1) p[1] = o.y;
    if (left > 2) p[2] = o.z;
    if (left > 3) p[3] = o.w;
  }
}
__device__ __forceinline__ void store_four(__nv_bfloat16* p, float4 v, Scale k, bool vec, int64_t left) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x * k.before * k.k, v.y * k.before * k.k);
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.z * k.before * k.k, v.w * k.before * k.k);
  if (vec) {
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    if (left > 0) p[0] = a.x;
    if (left > 1) p[1] = a.y;
    if (left > 2) p[2] = b.x;
    if (left > 3) p[3] = b.y;
  }
}

// The groups of the offsets in tiles of `width`; without offsets there is one
// group of all tokens, which the table holds only with ALWAYS.  False where the
// offsets are not valid.
template <bool ALWAYS>
__device__ __forceinline__ bool group_table(const GroupTable& t, const MatmulArgs& a, int width) {
  if (a.offsets != nullptr) {
    const bool ok = build_groups(t, a.offsets, a.groups, a.tokens, width);
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, GPTQ_ERR_INVALID_ARG);
    return ok;
  }
  if (ALWAYS) {
    if (threadIdx.x == 0) {
      t.off[0] = t.band[0] = t.tile[0] = 0;
      t.off[1] = static_cast<int>(a.tokens);
      t.band[1] = static_cast<int>((a.tokens + kFp4Band - 1) / kFp4Band);
      t.tile[1] = static_cast<int>((a.tokens + width - 1) / width);
    }
    __syncthreads();
  }
  return true;
}

// Items count token tiles first, then row tiles; the host has checked that
// there are less than 2^31.
template <bool ALWAYS>
__device__ __forceinline__ Tile tile_at(const GroupTable& t, const MatmulArgs& a, int wtiles, int width, uint32_t item) {
  Tile x;
  const int tt = static_cast<int>(item / wtiles);
  x.wtile = static_cast<int>(item - tt * wtiles);
  int first, last;
  if (!ALWAYS && a.offsets == nullptr) {
    x.g = 0;
    first = tt * width;
    x.token = first;
    last = static_cast<int>(a.tokens);
    x.xband = first / kFp4Band;
  } else {
    x.g = find_group(t.tile, a.groups, tt);
    first = (tt - t.tile[x.g]) * width;  // of the group's rows
    x.token = t.off[x.g] + first;
    last = t.off[x.g + 1];
    x.xband = t.band[x.g] + first / kFp4Band;
  }
  x.count = min(width, last - x.token);
  x.cols = (x.count + 15) / 16 * 16;
  x.xcol = first % kFp4Band / 32;
  return x;
}

// ---------------------------------------------------------------------------
// The kernel for few tokens: tiles of 128 weight rows x up to `width` tokens
// ---------------------------------------------------------------------------
//
// Bound by HBM: each weight is read once (128 * 4096 codes and their scales
// are 288 KB of nvfp4).  With about a tile an SM or more, one CTA an SM walks
// over the tiles with a ring of up to eight stages that never runs dry between
// two of them, in clusters of two that share the last tile of an odd number
// (64 tokens through 32 experts of 2048 x 4096, mxfp4: 30 us = 4.8 TB/s; from
// the first load to the last product it is 6.7 TB/s, the rest is the group
// table and the burst of first loads, 4 us, and the last tile's sums).  A
// layer with fewer tiles is cut along K: a cluster takes a tile, each of its
// CTAs a part of K, two CTAs an SM, and they then add up their sums in rank
// order, so the result does not depend on timing: of a few tokens each CTA
// sends its sums to the one that owns the token, as asynchronous stores that
// the owner's barrier counts; of many the owner reads them from the others
// (one token, 4096 x 4096: a CTA a tile 21 us, cut along K 6.5; the exchange
// through two cluster barriers and remote loads took 1 us more).
//
// RAW: X is not quantised yet (gptq_fp4_linear of a few tokens).  The epilogue
// warps then quantise the CTA's K range of its tokens into shared memory
// while the first weights arrive, which costs less than a launch in between
// (one token, 4096 x 4096, nvfp4: 8.3 us in two launches, 7.4 in one).

constexpr int kStreamThreads = 192;  // producer, MMA, 4 epilogue warps

// The epilogue warps' part of a RAW tile: x.count tokens, stages [k0, k1) of K,
// as B operand rows (128-byte swizzle) and scale tiles, stage by stage at
// `dst`.  Returns the tensor scale.  `src`: the tokens' rows of X, `red`: 4
// words.
template <bool BF16, bool NV>
__device__ __forceinline__ float quantize_tile(const QuantArgs& a, const Tile& x, int k0, int k1, uint8_t* dst, int* src,
                                               uint32_t* red) {
  using S = Fp4Lane<BF16, NV>;
  constexpr int kSize = BF16 ? 2 : 4, kAcross = kStageK / S::kLane;
  const int tid = threadIdx.x - 64;
  auto sync = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
  if (tid < x.count) src[tid] = source_row(a, x.token + tid);
  sync();
  const char* X = static_cast<const char*>(a.X);
  Unit u{1.0f, 1.0f, 1.0f, true};
  if (NV) {
    float t;
    if (a.given) {
      t = a.tensor_scale[x.g];
    } else {
      const int across = (a.n + S::kLane - 1) / S::kLane;
      uint32_t m = thread_max<BF16, 0, 4>(a, tid, 128, x.count * across, [&](int i, int& left) -> const char* {
        const int r = i / across, col = (i - r * across) * S::kLane, row = src[r];
        left = a.n - col;
        return row < 0 ? nullptr : X + (row * a.ldx + col) * kSize;
      });
      m = __reduce_max_sync(0xffffffffu, m);
      if (tid % 32 == 0) red[tid / 32] = m;
      sync();
      m = max(max(red[0], red[1]), max(red[2], red[3]));
      t = fmaxf(__fdiv_rn(__uint_as_float(m), 2688.0f), FLT_MIN);
    }
    u = unit_of(t);
  }
  const int wide = (k1 - k0) * kAcross;  // a multiple of 32 or 16, so a block's lanes stay together
  for (int i0 = 0; i0 < x.count * wide; i0 += 128) {
    const int i = i0 + tid, r = i / wide, c = i - r * wide;
    const bool in = r < x.count;
    const int col = k0 * kStageK + c * S::kLane, left = a.n - col;
    const int row = in ? src[r] : -1;
    const char* p = row < 0 || left <= 0 ? nullptr : X + (row * a.ldx + col) * kSize;
    uint32_t w[8];
    if (p != nullptr) {
      load_lane<BF16, 0>(p, left, col, w);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 0;
    }
    uint32_t codes[S::kLane / 8], byte;
    float s;
    quantize_lane<BF16, NV>(w, p, left, u, codes, byte, s);
    if (in) {
      uint8_t* stage = dst + c / kAcross * kRawStageBytes;
      const int at = c % kAcross * (S::kLane / 2);  // byte of the row's 128
      uint8_t* d = stage + r * (kStageK / 2) + ((at / 16) ^ (r % 8)) * 16 + at % 16;
      if (BF16)
        *reinterpret_cast<uint2*>(d) = make_uint2(codes[0], codes[S::kLane / 8 - 1]);
      else
        *reinterpret_cast<uint32_t*>(d) = codes[0];
      const int b = c % kAcross / S::kLanes;  // block of the stage; past the row's end it has scale 0
      if (c % S::kLanes == 0)
        stage[kRawTokens * (kStageK / 2) + b / 4 * kFp4TileBytes + r * 16 + b % 4] = static_cast<uint8_t>(left > 0 ? byte : 0);
    }
  }
  fence_proxy_async();  // the tensor cores and their copies read it
  return u.t;
}

// RAW: 0 X is quantised; 1 bf16, 2 fp32 X of q.  WALK: the CTAs walk over the
// tiles; without, a cluster has one tile (and no table of a single group).
template <bool NV, typename OUT, int RAW, bool WALK>
__global__ void __launch_bounds__(kStreamThreads, 2)
    fp4_stream_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, MatmulArgs a,
                      StreamShape shape, QuantArgs q) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = stream_stage_bytes(shape.width, RAW != 0);
  const int bbytes = RAW ? 0 : stage_bytes - kABytes - 2 * kSfBytes;  // of a stage's tokens, before its scales
  const int apart = stream_apart_bytes(shape.width, shape.splits);
  uint8_t* collect = apart > 0 ? smem + shape.stages * stage_bytes : smem;
  uint8_t* raw = smem + shape.stages * stage_bytes + apart;
  uint64_t* full = reinterpret_cast<uint64_t*>(raw + (RAW ? shape.raw_stages * kRawStageBytes : 0));
  uint64_t* empty = full + kStreamMaxStages;
  uint64_t* acc_full = empty + kStreamMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* sums_in = acc_empty + 2;  // the cluster's sums for this CTA's tokens have arrived
  uint64_t* x_ready = sums_in + 1;    // RAW: the tokens are quantised
  uint64_t* drain = x_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* raw_src = reinterpret_cast<int*>(tmem_slot + 2);                   // kRawTokens
  uint32_t* raw_red = reinterpret_cast<uint32_t*>(raw_src + kRawTokens);  // 4
  int* table = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + kStreamBarBytes);
  const GroupTable t{table, table + a.groups + 1, table + 2 * (a.groups + 1)};

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);
  const int lane = threadIdx.x % 32;
  constexpr int kBlk = NV ? 16 : 32;
  constexpr int kStageQuads = kStageK / (4 * kBlk);
  constexpr int kQuadMmas = kBlk / 16;
  constexpr uint32_t kStageSf = kStageQuads * kFp4TileBytes;
  const uint32_t tmem_cols = stream_tmem_cols(shape.width, WALK ? 2 : 1, shape.stages);

  if (threadIdx.x == 0) {
    for (int s = 0; s < shape.stages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + b, 1);
      mbar_init(acc_empty + b, 4);
    }
    mbar_init(sums_in, 1);
    mbar_init(x_ready, 128);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&wmap);
    if (!RAW) prefetch_tensormap(&xmap);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // (the cluster's barriers exist once all have arrived; waited for before the first use across it)
  if (shape.splits > 1) cluster_arrive();
  pdl_trigger();
  if (RAW || !a.early) pdl_wait();
  const bool ok_groups = group_table<WALK>(t, a, shape.width);
  const int wtiles = static_cast<int>((a.rows + kRows - 1) / kRows);
  // (uniform: see the pair kernel)
  const uint32_t token_tiles = WALK || a.offsets != nullptr ? uniform(t.tile[a.groups])
                                                            : static_cast<int>((a.tokens + shape.width - 1) / shape.width);
  const uint32_t items = ok_groups ? token_tiles * wtiles : 0;
  // This cluster's tiles are items `cluster`, + clusters, ...: `whole` of them
  // by single CTAs in turn, then what is left (`last`, one tile) by all of its
  // CTAs, each a part of K.
  const uint32_t clusters = gridDim.x / shape.splits, cluster = blockIdx.x / shape.splits;
  const int rank = blockIdx.x % shape.splits;
  const uint32_t mine_all = cluster >= items ? 0 : WALK ? (items - cluster + clusters - 1) / clusters : 1;
  const uint32_t whole_tiles = WALK ? mine_all / shape.splits * shape.splits : 0;
  constexpr int kAccs = WALK ? 2 : 1;
  const bool last = mine_all > whole_tiles;
  const int quads = fp4_quads(a.n, NV);
  const int mmas = (a.n + 63) / 64;
  const int kstages = (a.n + kStageK - 1) / kStageK;
  const int k0 = kstages * rank / shape.splits, k1 = kstages * (rank + 1) / shape.splits;  // of the last tile

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, a.wait_ns, abort_flag, a.status);
  };
  // this CTA's tiles, as m: rank, rank + splits, ... below whole_tiles, then the last one
  constexpr uint32_t kEnd = 0xffffffffu;
  const uint32_t after = last ? whole_tiles : kEnd;
  const uint32_t first_m = static_cast<uint32_t>(rank) < whole_tiles ? rank : after;
  auto next_m = [&](uint32_t m) {
    if (m >= whole_tiles) return kEnd;
    m += shape.splits;
    return m < whole_tiles ? m : after;
  };
  // the cluster's m-th tile
  auto tile_of = [&](uint32_t m) { return tile_at<WALK>(t, a, wtiles, shape.width, WALK ? cluster + m * clusters : cluster); };

  if (mine_all > 0) {
    // (the same in all CTAs of the cluster)
    const bool push = last && tile_of(whole_tiles).count <= kPushTokens;
    if (warp == 0) {
      if (elect_one()) {
        // ---------------- producer ----------------
        struct {
          int wy, token, boxes;
          const uint8_t* wsc;
          const uint8_t* xsc;
        } src;
        uint32_t m;
        int kb, kend;
        auto take = [&] {
          kb = m < whole_tiles ? 0 : k0;
          kend = m < whole_tiles ? kstages : k1;
          const Tile x = tile_of(m);
          src.wy = static_cast<int>(x.g * a.rows) + x.wtile * kRows;
          src.token = x.token;
          src.boxes = RAW ? 0 : (x.cols + kBoxRows - 1) / kBoxRows;
          src.wsc = a.wscales + (static_cast<int64_t>(x.g) * wtiles + x.wtile) * quads * kFp4TileBytes;
          src.xsc = a.xscales + static_cast<int64_t>(x.xband) * quads * kFp4TileBytes;
        };
        auto start = [&] {
          m = first_m;
          take();
        };
        auto next = [&] {
          if (++kb == kend) {
            m = next_m(m);
            if (m != kEnd) take();
          }
        };
        auto load_w = [&](uint32_t stage) {
          uint8_t* sa = smem + stage * stage_bytes;
          const uint32_t sf_bytes = min(kStageQuads, quads - kb * kStageQuads) * kFp4TileBytes;
          mbar_arrive_expect_tx(full + stage, kABytes + src.boxes * kBoxBytes + (RAW ? 1 : 2) * sf_bytes);
          tma_load_2d(sa, &wmap, full + stage, kb * (kStageK / 2), src.wy);
          bulk_load(sa + kABytes + bbytes, src.wsc + static_cast<int64_t>(kb) * kStageSf, sf_bytes, full + stage);
        };
        auto load_x = [&](uint32_t stage) {
          if (RAW) return;
          uint8_t* sa = smem + stage * stage_bytes;
          const uint32_t sf_bytes = min(kStageQuads, quads - kb * kStageQuads) * kFp4TileBytes;
          for (int b = 0; b < src.boxes; ++b)
            tma_load_2d(sa + kABytes + b * kBoxBytes, &xmap, full + stage, kb * (kStageK / 2), src.token + b * kBoxRows);
          bulk_load(sa + kABytes + bbytes + kStageSf, src.xsc + static_cast<int64_t>(kb) * kStageSf, sf_bytes, full + stage);
        };
        // the ring's first round: W before X is there
        uint32_t issued = 0;
        const uint32_t ring_stages = shape.stages;
        for (start(); issued < ring_stages && m != kEnd; ++issued, next()) load_w(issued);
        if (!RAW && a.early) pdl_wait();
        start();
        for (uint32_t i = 0; i < issued; ++i, next()) load_x(i);
        uint32_t stage = 0, phase = 1;
        for (; m != kEnd; next(), ++issued) {
          if (!wait(empty + stage, phase ^ 1u)) break;
          load_w(stage);
          load_x(stage);
          if (++stage == ring_stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        // every stage that was armed has received its bytes: the last use of each
        for (uint32_t u = issued > ring_stages ? issued - ring_stages : 0; u < issued; ++u)
          if (!mbar_wait(full + u % ring_stages, u / ring_stages & 1u, kDrainNs)) set_status(a.status, GPTQ_ERR_TIMEOUT);
      }
    } else if (warp == 1) {
      if (elect_one()) {
        // ---------------- MMA issuer ----------------
        uint32_t stage = 0, phase = 0, turn = 0;
        const uint32_t ring = smem_u32(smem);
        const uint32_t pair_bits = fp4_idesc(NV, 1, 0, 1) ^ fp4_idesc(NV, 1, 0, 0);
        const uint32_t sf_col = tmem + kAccs * shape.width;
        const int whole = mmas / (kStageK / 64);
        bool ok = !RAW || wait(x_ready, 0u);
        for (uint32_t m = first_m; ok && m != kEnd; m = next_m(m), ++turn) {
          const Tile x = tile_of(m);
          const int kbeg = m < whole_tiles ? 0 : k0, kend = m < whole_tiles ? kstages : k1;
          const uint32_t idesc = fp4_idesc(NV, 1, x.cols, 0);
          const uint32_t buf = WALK ? turn & 1u : 0u, acc = tmem + buf * shape.width;
          // (turn 0 and 1 find their accumulators empty)
          if (WALK && turn >= 2 && !(ok = wait(acc_empty + buf, (turn / 2 - 1) & 1u))) break;
          for (int kb = kbeg; kb < kend; ++kb) {
            if (!(ok = wait(full + stage, phase))) break;
            tc_fence_after();
            const uint32_t sa = ring + stage * stage_bytes;
            const uint32_t sb = RAW ? smem_u32(raw) + (kb - kbeg) * kRawStageBytes : sa + kABytes;
            const uint32_t ssa = sa + kABytes + bbytes, ssb = RAW ? sb + kRawTokens * (kStageK / 2) : ssa + kStageSf;
            // each ring stage has its own scale columns, 16 of W's and 16 of X's:
            // the stage is full again only after the products that read them
            const uint32_t tsa = sf_col + stage * 32, tsb = tsa + 16, tsx = tsb + x.xcol;
            const uint64_t adesc = smem_desc_sw128(sa, 16, 1024), bdesc = smem_desc_sw128(sb, 16, 1024);
            if (kb < whole) {
#pragma unroll
              for (int i = 0; i < kStageQuads; ++i) {
                copy_scales<1>(tsa + 4 * i, ssa + i * kFp4TileBytes);
                copy_scales<1>(tsb + 4 * i, ssb + i * kFp4TileBytes);
              }
#pragma unroll
              for (int i = 0; i < kStageK / 64; ++i)
                mma_fp4<NV, 1>(acc, adesc + 2 * i, bdesc + 2 * i, i % kQuadMmas ? idesc | pair_bits : idesc,
                               tsa + i / kQuadMmas * 4, tsx + i / kQuadMmas * 4, i > 0 || kb > kbeg);
            } else {
              const int q = quads - kb * kStageQuads, left = mmas - kb * (kStageK / 64);
              for (int i = 0; i < q; ++i) {
                copy_scales<1>(tsa + 4 * i, ssa + i * kFp4TileBytes);
                copy_scales<1>(tsb + 4 * i, ssb + i * kFp4TileBytes);
              }
              for (int i = 0; i < left; ++i)
                mma_fp4<NV, 1>(acc, adesc + 2 * i, bdesc + 2 * i, i % kQuadMmas ? idesc | pair_bits : idesc,
                               tsa + i / kQuadMmas * 4, tsx + i / kQuadMmas * 4, i > 0 || kb > kbeg);
            }
            mma_commit(empty + stage);
            if (++stage == static_cast<uint32_t>(shape.stages)) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (ok) mma_commit(acc_full + buf);
        }
        mma_commit(drain);
        if (!mbar_wait(drain, 0u, kDrainNs)) set_status(a.status, GPTQ_ERR_TIMEOUT);
      }
    } else {
      // ---------------- epilogue ----------------
      const int quad = warp & 3;  // the tensor-memory lanes of this warp
      const int f = quad * 32 + lane;
      if (!RAW && a.early) pdl_wait();
      uint32_t turn = 0;
      bool going = true;
      for (uint32_t m = rank; m < whole_tiles; m += shape.splits, ++turn) {
        const Tile x = tile_of(m);
        const float tx = a.xt != nullptr ? a.xt[x.g] : 1.0f;
        const Scale k = make_scale(a.wt != nullptr ? a.wt[x.g] : 1.0f, tx);
        const int64_t r = static_cast<int64_t>(x.wtile) * kRows + f;
        OUT* out = static_cast<OUT*>(a.y) + static_cast<int64_t>(x.token) * a.ldy + r;
        const uint32_t buf = WALK ? turn & 1u : 0u;
        int ok = 1;
        if (lane == 0) ok = wait(acc_full + buf, turn / 2 & 1u);
        if (!__shfl_sync(0xffffffffu, ok, 0)) {
          going = false;
          break;
        }
        tc_fence_after();
        const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * shape.width;
#pragma unroll 1
        for (int c = 0; c < x.count; c += 16) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(acc + c, v);
          tmem_ld_wait();
          if (r < a.rows) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c + j < x.count)
                store_out(out + static_cast<int64_t>(c + j) * a.ldy, __uint_as_float(v[j]) * k.before * k.k);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + buf);
      }
      if (last) {
        const Tile x = tile_of(whole_tiles);
        float tx = a.xt != nullptr ? a.xt[x.g] : 1.0f;
        if (RAW) {
          tx = quantize_tile<RAW == 1, NV>(q, x, k0, k1, raw, raw_src, raw_red);
          mbar_arrive(x_ready);
        }
        const Scale k = make_scale(a.wt != nullptr ? a.wt[x.g] : 1.0f, tx);
        const int64_t r = static_cast<int64_t>(x.wtile) * kRows + f;
        OUT* out = static_cast<OUT*>(a.y) + static_cast<int64_t>(x.token) * a.ldy + r;
        const uint32_t buf = WALK ? turn & 1u : 0u;
        const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * shape.width;
        int ok = going;
        if (lane == 0 && going) ok = wait(acc_full + buf, turn / 2 & 1u);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        tc_fence_after();
        // Token j belongs to rank j % splits, where it is row j / splits.  (A
        // CTA that gave up passes on what its accumulator holds, as the others
        // wait for it; the status word says that the result is not one.)
        const int mine = (x.count - rank + shape.splits - 1) / shape.splits;
        const int rows_each = (x.count + shape.splits - 1) / shape.splits;
        if (push && warp == 2 && lane == 0) mbar_arrive_expect_tx(sums_in, mine * shape.splits * kRows * 4);
        __syncwarp();
        cluster_wait();  // every CTA's barriers exist
        if (push) {
          if (apart == 0) {  // the other CTAs' rings are free
            cluster_arrive();
            cluster_wait();
          }
          // the sums of source rank q stand at [q][row][feature]
          const uint32_t at = smem_u32(collect) + (rank * rows_each * kRows + f) * 4, bar = smem_u32(sums_in);
          uint32_t v[16];
          tmem_ld_32x32b_x16(acc, v);
          tmem_ld_wait();
          int owner = 0, row = 0;
#pragma unroll
          for (int j = 0; j < kPushTokens; ++j) {
            if (j < x.count) st_async(at + row * kRows * 4, bar, owner, v[j]);
            if (++owner == shape.splits) {
              owner = 0;
              ++row;
            }
          }
          cluster_arrive();
          if (lane == 0) ok = wait(sums_in, 0u) && ok;
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (ok && r < a.rows) {
            const float* sums = reinterpret_cast<const float*>(collect) + f;
            for (int j = 0; j < mine; ++j) {
              float v = sums[j * kRows];
#pragma unroll
              for (int p = 1; p < 8; ++p)
                if (p < shape.splits) v += sums[(p * rows_each + j) * kRows];
              store_out(out + static_cast<int64_t>(j * shape.splits + rank) * a.ldy, v * k.before * k.k);
            }
          }
        } else {
          // this CTA's sums at [token][feature]; then a warp a token, a lane
          // four features, four tokens in flight
          float* sums = reinterpret_cast<float*>(collect) + f;
#pragma unroll 1
          for (int c = 0; c < x.count; c += 16) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(acc + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c + j < x.count) sums[(c + j) * kRows] = __uint_as_float(v[j]);
          }
          cluster_arrive();
          cluster_wait();
          const int64_t r4 = static_cast<int64_t>(x.wtile) * kRows + 4 * lane;
          OUT* o4 = static_cast<OUT*>(a.y) + static_cast<int64_t>(x.token) * a.ldy + r4;
          const bool vec = r4 + 4 <= a.rows && a.ldy % 4 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0;
          const int step = 4 * shape.splits;  // the cluster's epilogue warps
          for (int j0 = 4 * rank + warp - 2; j0 < x.count; j0 += 4 * step) {
            float4 v[4];
#pragma unroll
            for (int p = 0; p < 8; ++p) {
              if (p < shape.splits) {
                const uint32_t peer = smem_cluster_addr(collect, p) + 16 * lane;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                  if (j0 + w * step < x.count) {
                    const float4 z = ld_cluster_f32x4(peer + (j0 + w * step) * kRows * 4);
                    v[w] = p == 0 ? z : make_float4(v[w].x + z.x, v[w].y + z.y, v[w].z + z.z, v[w].w + z.w);
                  }
              }
            }
#pragma unroll
            for (int w = 0; w < 4; ++w)
              if (j0 + w * step < x.count) store_four(o4 + static_cast<int64_t>(j0 + w * step) * a.ldy, v[w], k, vec, a.rows - r4);
          }
          cluster_arrive();
        }
        cluster_wait();  // no CTA leaves while another may still use its memory
        // (after a wait that ran out: nor while sums that were sent are on their way)
        if (push && !ok && lane == 0) mbar_wait(sums_in, 0u, kDrainNs);
        __syncwarp();
      }
      tc_fence_before();
    }
    __syncwarp();
    if (last && warp < 2) {  // the barriers of the epilogue
      cluster_wait();
      if (!push || apart == 0) {
        cluster_arrive();
        cluster_wait();
      }
      cluster_arrive();
      cluster_wait();
    }
  }
  if (shape.splits > 1 && !last) cluster_wait();
  if (!RAW && a.early) pdl_wait();  // (in every CTA: this kernel does not end before the quantiser)
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
}

// ---------------------------------------------------------------------------
// The kernel for many tokens: CTA pairs, 256 weight rows x up to 256 tokens
// ---------------------------------------------------------------------------
//
// Bound by shared memory and the tensor cores: a stage of 256 columns brings
// 38 KB to each CTA, which the products and scale copies read again, 76 KB at
// 128 bytes a cycle = 608 cycles; measured 610 to 625 cycles a stage.  Its four
// products of 256 x 256 x 64 keep the tensor pipe for 4 x 131 of them (counted:
// about 520); alone, its twelve scale copies take 10 each, so they overlap products
// or each other, as 644 in line would be more than measured.  A tile of one CTA (128 x 256) would move 108 KB.  The
// accumulators of two tiles overlap, as two of 256 columns and the scales do
// not fit: the next tile's products wait until the epilogue has read the
// overlap, about 850 cycles.  8192 tokens, 11008 x 4096, nvfp4, bf16 out: 148 us
// = 5.0 PFLOP/s, 3.0 times the card's bf16 rate (170 us when it is kept at it:
// the clock falls to 1.5 GHz under the power limit).  Steps on the way: one
// CTA a tile 487 us; pairs and overlapped accumulators 390; loops run by whole
// warps 242; whole stages issued without conditions 181 (a branch around each
// instruction cost more than the instruction); single-thread roles and a
// rolled epilogue 163; an arrival that does not wait for the epilogue's own
// stores 158; the epilogue through stmatrix and TMA stores 148.

constexpr int kPairRows = 256;
constexpr int kPairStages = 5;
constexpr int kPairBBytes = kTokens / 2 * kStageK / 2;  // this CTA's half of the tokens
constexpr int kPairStageBytes = kABytes + kPairBBytes + 3 * kSfBytes;
constexpr int kPairEpiWarps = 8;
constexpr int kPairThreads = 64 + 32 * kPairEpiWarps;
constexpr int kStageOutBytes = 32 * 64;  // a warp's 32 tokens x 32 features in bf16
constexpr size_t kPairSmemBytes = 1024 + size_t(kPairStages) * kPairStageBytes + kPairEpiWarps * kStageOutBytes + 256;
// Tensor memory: two accumulators that overlap in columns [96, 256), and three
// sets of scales (16 columns of W's, 32 of X's).  The epilogue empties the
// overlap first.
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kAccShift = 96;
constexpr uint32_t kPairSfCol = kAccShift + kTokens, kPairSfStride = 48, kPairSfSets = 3;
static_assert(kPairSfCol + kPairSfSets * kPairSfStride <= kTmemCols, "tensor memory");

// A warp's block of 32 features x 32 tokens, from tensor memory to y.  TMA
// (bf16): read as matrix fragments, transposed by stmatrix into rows of 64
// bytes (32 features of a token, 64-byte swizzle) and written by a TMA store;
// the end of a group's rows or of W's (a TMA store is cut at 16 bytes, not at
// an element) row by row.  Else: a lane a feature, row by row.
struct Out {
  const CUtensorMap* map;
  uint8_t* stg;      // this warp's 2 KB
  int64_t ldy;
};

// store(row, j) for `last` rows, N at most; the pointer runs with them.  (The
// epilogue is bound by its instructions: with an address made of j and a test
// for each row, 28 of them to a row, 4614 tokens x 779 -> 3328 in fp32 took 35.7
// us instead of 20.7.)
template <int N, typename T, typename F>
__device__ __forceinline__ void rows_of(T* row, int64_t step, int last, F store) {
  if (last >= N) {
#pragma unroll
    for (int j = 0; j < N; ++j, row += step) store(row, j);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j, row += step) {
      if (j >= last) break;
      store(row, j);
    }
  }
}

template <typename OUT, bool TMA>
struct Block {
  static __device__ __forceinline__ void load(uint32_t taddr, uint32_t (&v)[32]) { tmem_ld_32x32b_x32(taddr, v); }
  static __device__ __forceinline__ void store(uint32_t (&v)[32], Scale k, const Out& o, OUT* y, int, int, int tokens,
                                               int64_t features) {
    const int lane = threadIdx.x & 31;
    if (k.before != 1.0f) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * k.before);
    }
    if (lane < features)
      rows_of<32>(y + lane, o.ldy, tokens, [&](OUT* q, int j) { store_out(q, __uint_as_float(v[j]) * k.k); });
  }
};

template <>
struct Block<__nv_bfloat16, true> {
  static __device__ __forceinline__ void load(uint32_t taddr, uint32_t (&v)[32]) {
    tmem_ld_16x256b_x4(taddr, v);
    tmem_ld_16x256b_x4(taddr + (16u << 16), v + 16);
  }
  static __device__ __forceinline__ void store(uint32_t (&v)[32], Scale k, const Out& o, __nv_bfloat16* y, int token,
                                               int feature, int tokens, int64_t features) {
    const int lane = threadIdx.x & 31;
    if (k.before != 1.0f) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * k.before);
    }
    uint32_t p[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(v[2 * j]) * k.k, __uint_as_float(v[2 * j + 1]) * k.k);
      p[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    if (lane == 0) bulk_wait_read();  // the last block's store has read the buffer
    __syncwarp();
    const uint32_t at = smem_u32(o.stg) + (lane % 8) * 64;  // row 8 i + lane % 8, matrix (feature eight) lane / 8
    const uint32_t swz = ((lane / 8) ^ (lane / 2 % 4)) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) stmatrix_x4_trans(at + 512 * i + swz, p[2 * i], p[2 * i + 1], p[8 + 2 * i], p[8 + 2 * i + 1]);
    if (tokens >= 32 && features >= 32) {
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(o.map, o.stg, feature, token);
        bulk_commit();
      }
    } else {
      __syncwarp();
      if (lane < features) {
        const uint8_t* from = o.stg + 2 * (lane % 8);
        __nv_bfloat16* row = y + lane;
#pragma unroll 1
        for (int left = min(tokens, 32); left > 0; left -= 8, from += 512) {
          uint16_t u[8];  // (read before the first is written: the compiler cannot know that they are not the same)
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] = *reinterpret_cast<const uint16_t*>(from + 16 * ((lane / 8) ^ (j / 2)) + 64 * j);
#pragma unroll
          for (int j = 0; j < 8; ++j, row += o.ldy)
            if (j < left) *reinterpret_cast<uint16_t*>(row) = u[j];
        }
      }
      __syncwarp();
    }
  }
};

// Boxes of 32 token rows that a CTA of a pair loads for a tile of `cols`
// tokens: 0 stands for one box of 128 rows, where boxes of 32 load no less.
__device__ __forceinline__ int pair_boxes(int cols) { return cols / 2 > 96 ? 0 : (cols / 2 + kBoxRows - 1) / kBoxRows; }
// Bytes that a CTA of a pair loads a stage; `scales` of 128 rows.
__device__ __forceinline__ uint32_t pair_bytes(int boxes, uint32_t scales) {
  return kABytes + (boxes == 0 ? kPairBBytes : boxes * kBoxBytes) + 3 * scales;
}
// The same of an item's stages.  (Out of line: only the end of a run whose waits
// ran out asks for it.)
static __device__ __noinline__ uint32_t pair_item_bytes(const int* off, const int* tile, int groups, int wtiles, int width,
                                                        uint32_t item, uint32_t scales) {
  const int tt = static_cast<int>(item / wtiles), g = find_group(tile, groups, tt);
  const int count = min(width, off[g + 1] - off[g] - (tt - tile[g]) * width);
  return pair_bytes(pair_boxes((count + 15) / 16 * 16), scales);
}

// WIDTH: tokens of a tile, 256 or 128.  TMA: y is written by TMA.
template <bool NV, typename OUT, int WIDTH, bool TMA>
__global__ void __launch_bounds__(kPairThreads, 1)
    fp4_pair_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                    const __grid_constant__ CUtensorMap xwide, const __grid_constant__ CUtensorMap wsmap,
                    const __grid_constant__ CUtensorMap xsmap, const __grid_constant__ CUtensorMap ymap, MatmulArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + size_t(kPairStages) * kPairStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kPairEpiWarps * kStageOutBytes);
  uint64_t* empty = full + kPairStages;
  uint64_t* acc_full = empty + kPairStages;  // one: a tile's products are complete
  uint64_t* acc_free = acc_full + 1;         // the overlap of a tile's accumulator has been read
  uint64_t* drain = acc_free + 1;
  uint64_t* odd_done = drain + 1;            // of the even CTA: the odd one's producer has stopped, after *odd_issued stages
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(odd_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* odd_issued = tmem_slot + 2;
  int* table = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + 256);
  const GroupTable t{table, table + a.groups + 1, table + 2 * (a.groups + 1)};

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);  // the same register for the whole warp
  const int lane = threadIdx.x % 32;
  const uint32_t rank = uniform(cluster_ctarank());
  const uint32_t pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  constexpr int kBlk = NV ? 16 : 32;
  constexpr int kStageQuads = kStageK / (4 * kBlk);
  constexpr int kQuadMmas = kBlk / 16;
  constexpr uint32_t kStageSf = kStageQuads * kFp4TileBytes;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(full + s, 1);   // the even CTA's expect-tx arrival (and both CTAs' bytes)
      mbar_init(empty + s, 1);  // a commit each use
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_free, 2 * kPairEpiWarps);  // the epilogue warps of both CTAs
    mbar_init(drain, 1);
    mbar_init(odd_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    if (rank == 0) mbar_arrive_expect_tx(odd_done, 4);
    prefetch_tensormap(&wmap);
    prefetch_tensormap(&xmap);
    prefetch_tensormap(&xwide);
    prefetch_tensormap(&wsmap);
    prefetch_tensormap(&xsmap);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before either is used across the pair
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  pdl_trigger();
  if (!a.early) pdl_wait();
  const bool ok_groups = group_table<true>(t, a, WIDTH);
  if (a.early) pdl_wait();
  const int wtiles = static_cast<int>((a.rows + kPairRows - 1) / kPairRows);
  const int wbands = static_cast<int>((a.rows + kRows - 1) / kRows);
  // (read from the table by every lane and passed through `uniform`: the
  // compiler then knows the loops' end to be the same for the whole warp and
  // keeps descriptors in uniform registers.  With the end chosen between the
  // table and the arguments a stage took the MMA thread four times as long to
  // issue, and 8192 x 4096 -> 11008 took 271 us instead of 148.)
  const uint32_t items = ok_groups ? static_cast<uint32_t>(uniform(t.tile[a.groups])) * wtiles : 0;
  const int quads = fp4_quads(a.n, NV);
  const int mmas = (a.n + 63) / 64;
  const int kstages = (a.n + kStageK - 1) / kStageK;

  auto tile_of = [&](uint32_t item) { return tile_at<true>(t, a, wtiles, WIDTH, item); };
  // A single thread's wait.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, a.wait_ns, abort_flag, a.status);
  };

  if (warp == 0) {
    if (elect_one()) {
      // ---------------- producer (both CTAs) ----------------
      uint32_t stage = 0, phase = 0, issued = 0;
      const uint32_t full0 = smem_cluster_addr(full, 0);  // the even CTA's barriers
      bool ok = true;
      for (uint32_t item = pair; ok && item < items; item += pairs) {
        const Tile x = tile_of(item);
        const int half = x.cols / 2;  // tokens of this CTA
        const int boxes = pair_boxes(x.cols);
        const uint32_t bytes = 2 * pair_bytes(boxes, kStageSf);
        // the odd CTA's rows may not exist: it then loads the last band's scales for nothing
        const int wband = x.g * wbands + min(2 * x.wtile + static_cast<int>(rank), wbands - 1);
        const int xband = x.xband;
        const int wy = static_cast<int>(x.g * a.rows) + x.wtile * kPairRows + static_cast<int>(rank) * kRows;
        const int xy = x.token + static_cast<int>(rank) * half;
        for (int kb = 0; kb < kstages; ++kb) {
          ok = wait(empty + stage, phase ^ 1u);
          if (!ok) break;
          uint8_t* sa = smem + stage * kPairStageBytes;
          const uint32_t bar = full0 + 8 * stage;
          if (rank == 0) mbar_arrive_expect_tx(full + stage, bytes);
          tma_load_2d_pair(sa, &wmap, bar, kb * (kStageK / 2), wy);
          if (boxes == 0)
            tma_load_2d_pair(sa + kABytes, &xwide, bar, kb * (kStageK / 2), xy);
          else
            for (int b = 0; b < boxes; ++b)
              tma_load_2d_pair(sa + kABytes + b * kBoxBytes, &xmap, bar, kb * (kStageK / 2), xy + b * kBoxRows);
          tma_load_3d_pair(sa + kABytes + kPairBBytes, &wsmap, bar, 0, kb * kStageQuads, wband);
          tma_load_3d_pair(sa + kABytes + kPairBBytes + kStageSf, &xsmap, bar, 0, kb * kStageQuads, xband);
          ++issued;
          if (++stage == kPairStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      drain_pair(rank, issued, kPairStages, full, drain, odd_done, odd_issued, abort_flag, a.status, a.wait_ns, kDrainNs,
                 [&](uint32_t u) {
                   return pair_item_bytes(t.off, t.tile, a.groups, wtiles, WIDTH, pair + u / kstages * pairs, kStageSf);
                 });
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      // ---------------- MMA issuer (even CTA) ----------------
      // Per stage twelve scale copies (nvfp4) and four products.  Whole stages
      // take a path without conditions, as those are what issuing costs.
      uint32_t stage = 0, phase = 0, tiles = 0;
      uint32_t set = 0;                    // scale columns, in turn
      uint32_t late = 0, late_phase = 0;   // the stage whose products last read them
      uint32_t ahead = 0;                  // stages issued, up to the sets
      const uint32_t ring = smem_u32(smem);
      const uint32_t pair_bits = fp4_idesc(NV, 2, 0, 1) ^ fp4_idesc(NV, 2, 0, 0);
      const int whole = mmas / (kStageK / 64);
      // the overlap with the last tile's accumulator has been read (waited for
      // when the new tile's first scales are on their way)
      auto free_acc = [&](uint32_t tiles) {
        if (tiles > 0 && !wait(acc_free, (tiles - 1) & 1u)) return false;
        tc_fence_after();
        return true;
      };
      bool ok = true;
      for (uint32_t item = pair; ok && item < items; item += pairs, ++tiles) {
        const Tile x = tile_of(item);
        const uint32_t idesc = fp4_idesc(NV, 2, x.cols, 0);
        const uint32_t acc = tmem + (tiles & 1u) * kAccShift;
        for (int kb = 0; kb < kstages; ++kb) {
          if (ahead == kPairSfSets) {
            if (!(ok = wait(empty + late, late_phase))) break;
            if (++late == kPairStages) {
              late = 0;
              late_phase ^= 1u;
            }
          } else {
            ++ahead;
          }
          if (!(ok = wait(full + stage, phase))) break;
          tc_fence_after();
          const uint32_t sa = ring + stage * kPairStageBytes;
          const uint32_t ssa = sa + kABytes + kPairBBytes, ssb = ssa + kStageSf;
          const uint32_t tsa = tmem + kPairSfCol + set * kPairSfStride, tsb = tsa + 16;
          const uint64_t adesc = smem_desc_sw128(sa, 16, 1024), bdesc = smem_desc_sw128(sa + kABytes, 16, 1024);
          // 64 columns of K are 32 bytes, two units of a descriptor's address
          if (kb < whole) {
#pragma unroll
            for (int i = 0; i < kStageQuads; ++i) {
              copy_scales<2>(tsa + 4 * i, ssa + i * kFp4TileBytes);
              copy_scales<2>(tsb + 8 * i, ssb + i * kFp4TileBytes);
              copy_scales<2>(tsb + 8 * i + 4, ssb + kStageSf + i * kFp4TileBytes);  // (for nothing up to 128 tokens)
            }
            if (kb == 0 && !(ok = free_acc(tiles))) break;
#pragma unroll
            for (int i = 0; i < kStageK / 64; ++i)
              mma_fp4<NV, 2>(acc, adesc + 2 * i, bdesc + 2 * i, i % kQuadMmas ? idesc | pair_bits : idesc,
                             tsa + i / kQuadMmas * 4, tsb + i / kQuadMmas * 8, i > 0 || kb > 0);
          } else {
            const int q = quads - kb * kStageQuads, m = mmas - kb * (kStageK / 64);
            for (int i = 0; i < q; ++i) {
              copy_scales<2>(tsa + 4 * i, ssa + i * kFp4TileBytes);
              copy_scales<2>(tsb + 8 * i, ssb + i * kFp4TileBytes);
              copy_scales<2>(tsb + 8 * i + 4, ssb + kStageSf + i * kFp4TileBytes);
            }
            if (kb == 0 && !(ok = free_acc(tiles))) break;
            for (int i = 0; i < m; ++i)
              mma_fp4<NV, 2>(acc, adesc + 2 * i, bdesc + 2 * i, i % kQuadMmas ? idesc | pair_bits : idesc,
                             tsa + i / kQuadMmas * 4, tsb + i / kQuadMmas * 8, i > 0 || kb > 0);
          }
          mma_commit_pair(empty + stage, 0x3);
          set = set == kPairSfSets - 1 ? 0 : set + 1;
          if (++stage == kPairStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) mma_commit_pair(acc_full, 0x3);
      }
      mma_commit_pair(drain, 0x3);  // (the odd CTA leaves after it too)
      if (!mbar_wait(drain, 0u, kDrainNs)) set_status(a.status, GPTQ_ERR_TIMEOUT);
    }
  } else {
    // ---------------- epilogue (both CTAs) ----------------
    const int quad = warp & 3;            // the tensor-memory lanes of this warp
    const int turn = (warp - 2) >> 2;     // which of the two warps with these lanes
    const Out o{&ymap, staging + (warp - 2) * kStageOutBytes, a.ldy};
    uint32_t tiles = 0;
    for (uint32_t item = pair; item < items; item += pairs, ++tiles) {
      const Tile x = tile_of(item);
      int ok = 1;
      if (lane == 0) ok = wait(acc_full, tiles & 1u);
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      tc_fence_after();
      const int64_t r0 = static_cast<int64_t>(x.wtile) * kPairRows + rank * kRows + quad * 32;
      const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + (tiles & 1u) * kAccShift;
      // chunks of 32 tokens, those in the overlap first: columns [96, 256) of
      // the first accumulator, [0, 160) of the second
      const int first = (tiles & 1u ? 0 : 3) + turn;
      uint32_t v0[32], v1[32], v2[32];
      Block<OUT, TMA>::load(acc + first % 8 * 32, v0);
      Block<OUT, TMA>::load(acc + (first + 2) % 8 * 32, v1);
      Block<OUT, TMA>::load(acc + (first + 4) % 8 * 32, v2);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(smem_cluster_addr(acc_free, 0));
      const Scale k = tile_scale(a, x.g);
      OUT* out = static_cast<OUT*>(a.y) + static_cast<int64_t>(x.token) * a.ldy + r0;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {  // (rolled: the code of one block stays in the instruction cache)
        const int c = (first + 2 * i) % 8 * 32;
        if (c < x.count && r0 < a.rows)
          Block<OUT, TMA>::store(v0, k, o, out + c * a.ldy, x.token + c, static_cast<int>(r0), x.count - c, a.rows - r0);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          v0[j] = v1[j];
          v1[j] = v2[j];
        }
        if (i == 0) {
          Block<OUT, TMA>::load(acc + (first + 6) % 8 * 32, v2);
          tmem_ld_wait();
        }
      }
      tc_fence_before();
    }
    if (TMA && lane == 0) bulk_wait();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while the pair still uses its memory
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

template <bool NV, typename OUT, int RAW, bool WALK>
gptq_status launch_stream(const CUtensorMap& wmap, const CUtensorMap& xmap, const MatmulArgs& a, const StreamShape& s,
                          const QuantArgs& q, const DeviceInfo* info, cudaStream_t st) {
  static std::atomic<bool> attr_set[64] = {};  // per device, shared by host threads
  if (!attr_set[info->device]) {
    if (cudaFuncSetAttribute(fp4_stream_kernel<NV, OUT, RAW, WALK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kStreamMaxSmem)) != cudaSuccess)
      return GPTQ_ERR_CUDA;
    attr_set[info->device] = true;
  }
  const int64_t items = stream_tiles(s, a.tokens, a.groups, a.offsets != nullptr, a.rows);
  if (items * s.splits > INT32_MAX) return GPTQ_ERR_UNSUPPORTED;
  // clusters walk over the items, or have one each
  const int64_t ctas = s.splits * (s.accs == 2 ? std::min<int64_t>(items, std::max(1, info->sm_count / s.splits)) : items);
  const size_t smem = stream_smem(s, RAW != 0, a.groups);
  return launch_cluster_pdl(fp4_stream_kernel<NV, OUT, RAW, WALK>, static_cast<unsigned>(ctas), kStreamThreads, smem, s.splits,
                            st, wmap, xmap, a, s, q) == cudaSuccess
             ? launch_status()
             : GPTQ_ERR_CUDA;
}

template <bool NV, typename OUT, int WIDTH, bool TMA>
gptq_status launch_pair_of(const CUtensorMap& wmap, const CUtensorMap& xmap, const CUtensorMap& xwide,
                        const CUtensorMap& wsmap, const CUtensorMap& xsmap, const CUtensorMap& ymap, const MatmulArgs& a, const DeviceInfo* info,
                        cudaStream_t st) {
  static std::atomic<bool> attr_set[64] = {};  // per device, shared by host threads
  if (!attr_set[info->device]) {
    if (cudaFuncSetAttribute(fp4_pair_kernel<NV, OUT, WIDTH, TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kPairSmemBytes + table_bytes(kFp4MaxGroups))) != cudaSuccess)
      return GPTQ_ERR_CUDA;
    attr_set[info->device] = true;
  }
  const bool ragged = a.offsets != nullptr;
  // token tiles: each group's last one may be part full
  const int64_t tiles = ragged ? a.tokens / WIDTH + std::min<int64_t>(a.groups, a.tokens) : ceil_div(a.tokens, WIDTH);
  const int64_t items = tiles * ceil_div(a.rows, kPairRows);
  if (items > INT32_MAX - 2 * info->sm_count) return GPTQ_ERR_UNSUPPORTED;
  const unsigned grid = 2 * static_cast<unsigned>(std::min<int64_t>(items, std::max(1, info->sm_count / 2)));
  return launch_cluster_pdl(fp4_pair_kernel<NV, OUT, WIDTH, TMA>, grid, kPairThreads, kPairSmemBytes + table_bytes(a.groups), 2, st, wmap, xmap, xwide, wsmap,
                            xsmap, ymap, a) == cudaSuccess
             ? launch_status()
             : GPTQ_ERR_CUDA;
}

// Tiles of 128 tokens where those of 256 would leave half of the pairs idle
// (777 tokens, 1111 x 2000: a fifth less).
template <bool NV, typename OUT>
gptq_status launch_pair(const CUtensorMap& wmap, const CUtensorMap& xmap, const CUtensorMap& xwide,
                        const CUtensorMap& wsmap, const CUtensorMap& xsmap, const CUtensorMap& ymap, const MatmulArgs& a,
                        const DeviceInfo* info, cudaStream_t st) {
  if (a.offsets == nullptr && ceil_div(a.tokens, kTokens) * ceil_div(a.rows, kPairRows) * 4 <= info->sm_count)
    return launch_pair_of<NV, OUT, kTokens / 2, false>(wmap, xmap, xwide, wsmap, xsmap, ymap, a, info, st);
  return launch_pair_of<NV, OUT, kTokens, false>(wmap, xmap, xwide, wsmap, xsmap, ymap, a, info, st);
}

// Whether the pair kernel takes it.  Both are timed on nvfp4 products, in us:
//   rows x n, tokens       8     32    64    96    128   256
//   4096 x 4096   stream   6.5   7.7   9.5   11.0  12.4  12.8
//                 pair     9.7   9.4   9.6   9.8   10.0  10.6
//   4096 x 11008  stream   8.8   9.6   12.2  14.0  15.4  18.8
//                 pair     17.9  17.8  17.9  18.2  18.5  19.6
// The stream kernel pays for tokens (sums to exchange), the pair kernel, which
// does not cut K, for its depth.  Above 128 tokens it is the pair kernel, up to
// 64 the other, and between them the sums below, which are fitted to these
// times.  Groups: up to 32 tokens each, whatever rows, n and their number are.
// 32 of 2048 x 4096 take 32.7 and 34.2 us at 32 tokens each, 38.9 and 36.4 at
// 96; 8 of 2048 x 2048 8.5 and 8.6 at 8, 10.2 and 8.4 at 32, where the rule
// takes the slower one: it fits many groups, which read much of W, not few.
bool many_tokens(int64_t tokens, int groups, bool ragged, int64_t rows, int n, int sms) {
  if (ragged) return tokens > 32 * static_cast<int64_t>(groups);
  if (tokens <= 64 || tokens > kFp4Band) return tokens > kFp4Band;
  const int kstages = static_cast<int>(ceil_div(n, kStageK));
  const StreamShape s = stream_shape(tokens, groups, ragged, rows, n, sms);
  const int64_t tiles = ceil_div(rows, kRows) * (s.accs == 2 ? 1 : s.splits);
  const double stream = 5.5 + 0.04 * tokens + 0.43 * ceil_div(tiles, sms) * ceil_div(kstages, s.accs == 2 ? 1 : s.splits);
  const double pair = 4.5 + 0.31 * kstages * ceil_div(ceil_div(rows, kPairRows), std::max(1, sms / 2));
  return pair < stream;
}

// Scale tiles as bytes x quads x bands, `bands` bands a box.
bool scale_map(CUtensorMap* map, const uint8_t* scales, int64_t quads, int64_t bands, bool nv, uint32_t box_bands) {
  return make_tensor_map_3d(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, scales,
                            {kFp4TileBytes / 4, static_cast<uint64_t>(quads), static_cast<uint64_t>(bands)},
                            {kFp4TileBytes, static_cast<uint64_t>(quads) * kFp4TileBytes},
                            {kFp4TileBytes / 4, static_cast<uint32_t>(kStageK / (4 * fp4_block(nv))), box_bands},
                            CU_TENSOR_MAP_SWIZZLE_NONE);
}

}  // namespace

// A product's arguments but for X's.
static MatmulArgs product_args(const uint8_t* wscales, const float* wt, int groups, int64_t rows, int n, int64_t tokens,
                               const int32_t* offsets, void* y, int64_t ldy, const DeviceInfo* info) {
  MatmulArgs a = {};
  a.wscales = wscales;
  a.wt = wt;
  a.offsets = offsets;
  a.groups = groups;
  a.rows = rows;
  a.tokens = tokens;
  a.n = n;
  a.y = y;
  a.ldy = ldy;
  a.status = info->status;
  a.wait_ns = wait_limit_ns();
  return a;
}

static bool weight_map(CUtensorMap* map, const uint8_t* wq, int groups, int64_t rows, int n) {
  const int64_t pitch = fp4_pitch(n);
  return make_tensor_map_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, wq, pitch, static_cast<uint64_t>(groups) * rows, pitch,
                            kStageK / 2, kRows, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool fp4_linear_raw(int64_t tokens, int groups, bool ragged, int64_t rows, int n) {
  const DeviceInfo* info = device_info();
  StreamShape s;
  return info != nullptr && raw_shape(tokens, groups, ragged, rows, n, info->sm_count, &s);
}

// The product of a few tokens that it quantises itself (fp4_linear_raw).
gptq_status fp4_raw_matmul(bool nv, const uint8_t* wq, const uint8_t* wscales, const float* wt, int groups, int64_t rows,
                           int n, const void* X, int x_bf16, int64_t x_rows, int64_t ldx, const int32_t* row_index,
                           const float* x_tensor, int64_t tokens, const int32_t* offsets, void* y, int y_bf16, int64_t ldy,
                           cudaStream_t st) {
  const DeviceInfo* info = device_info();
  StreamShape s;
  CUtensorMap wmap;
  if (info == nullptr || !raw_shape(tokens, groups, offsets != nullptr, rows, n, info->sm_count, &s) ||
      !weight_map(&wmap, wq, groups, rows, n))
    return GPTQ_ERR_CUDA;
  const MatmulArgs a = product_args(wscales, wt, groups, rows, n, tokens, offsets, y, ldy, info);
  const QuantArgs q = fp4_quant_args(X, x_bf16, x_rows, n, ldx, row_index, tokens, offsets, groups, x_tensor != nullptr,
                                     const_cast<float*>(x_tensor), info->status);
  if (nv && x_bf16)
    return y_bf16 ? launch_stream<true, __nv_bfloat16, 1, false>(wmap, wmap, a, s, q, info, st)
                  : launch_stream<true, float, 1, false>(wmap, wmap, a, s, q, info, st);
  if (nv)
    return y_bf16 ? launch_stream<true, __nv_bfloat16, 2, false>(wmap, wmap, a, s, q, info, st)
                  : launch_stream<true, float, 2, false>(wmap, wmap, a, s, q, info, st);
  if (x_bf16)
    return y_bf16 ? launch_stream<false, __nv_bfloat16, 1, false>(wmap, wmap, a, s, q, info, st)
                  : launch_stream<false, float, 1, false>(wmap, wmap, a, s, q, info, st);
  return y_bf16 ? launch_stream<false, __nv_bfloat16, 2, false>(wmap, wmap, a, s, q, info, st)
                : launch_stream<false, float, 2, false>(wmap, wmap, a, s, q, info, st);
}

gptq_status fp4_matmul(bool nv, const uint8_t* wq, const uint8_t* wscales, const float* wt, int groups, int64_t rows,
                       int n, const uint8_t* xq, const uint8_t* xscales, const float* xt, int64_t tokens,
                       const int32_t* offsets, void* y, int y_bf16, int64_t ldy, bool early, cudaStream_t st) {
  const DeviceInfo* info = device_info();
  if (info == nullptr) return GPTQ_ERR_CUDA;
  const int64_t pitch = fp4_pitch(n);
  CUtensorMap wmap, xmap;
  if (!weight_map(&wmap, wq, groups, rows, n) ||
      !make_tensor_map_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, pitch, tokens, pitch, kStageK / 2, kBoxRows,
                          CU_TENSOR_MAP_SWIZZLE_128B))
    return GPTQ_ERR_CUDA;
  MatmulArgs a = product_args(wscales, wt, groups, rows, n, tokens, offsets, y, ldy, info);
  a.xscales = xscales;
  a.xt = xt;
  a.early = early;
  if (!many_tokens(tokens, groups, offsets != nullptr, rows, n, info->sm_count)) {
    const StreamShape s = stream_shape(tokens, groups, offsets != nullptr, rows, n, info->sm_count);
    const QuantArgs none = {};
    if (s.accs == 2) {
      if (nv)
        return y_bf16 ? launch_stream<true, __nv_bfloat16, 0, true>(wmap, xmap, a, s, none, info, st)
                      : launch_stream<true, float, 0, true>(wmap, xmap, a, s, none, info, st);
      return y_bf16 ? launch_stream<false, __nv_bfloat16, 0, true>(wmap, xmap, a, s, none, info, st)
                    : launch_stream<false, float, 0, true>(wmap, xmap, a, s, none, info, st);
    }
    if (nv)
      return y_bf16 ? launch_stream<true, __nv_bfloat16, 0, false>(wmap, xmap, a, s, none, info, st)
                    : launch_stream<true, float, 0, false>(wmap, xmap, a, s, none, info, st);
    return y_bf16 ? launch_stream<false, __nv_bfloat16, 0, false>(wmap, xmap, a, s, none, info, st)
                  : launch_stream<false, float, 0, false>(wmap, xmap, a, s, none, info, st);
  }
  const int64_t quads = fp4_quads(n, nv);
  const int64_t xbands = offsets != nullptr ? fp4_bands(tokens, groups, true) : ceil_div(tokens, kFp4Band);
  CUtensorMap wsmap, xsmap;
  if (!scale_map(&wsmap, wscales, quads, fp4_bands(groups * rows, groups, false), nv, 1) ||
      !scale_map(&xsmap, xscales, quads, xbands, nv, 2))
    return GPTQ_ERR_CUDA;
  CUtensorMap xwide, ymap = xmap;  // (ymap unused without TMA)
  if (!make_tensor_map_2d(&xwide, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, pitch, tokens, pitch, kStageK / 2, kTokens / 2,
                          CU_TENSOR_MAP_SWIZZLE_128B))
    return GPTQ_ERR_CUDA;
  // Stores by TMA where pairs walk over many tiles of one matrix: they take less
  // of shared memory's time from the products.  With a tile or less a pair, and
  // with groups, whose tiles end early, a lane a feature is faster.  (nvfp4 8192
  // x 4096 -> 11008: 150 us by TMA, 156 without; mxfp4 1555 x 2000 -> 4096 13.5
  // and 14.0, -> 1112 9.0 and 8.3; 32 groups of 125 and 250 tokens x 2000 ->
  // 2048 25.5 and 24.0, 34.2 and 32.2; groups of thousands were not timed.)
  const bool y_tma = y_bf16 && reinterpret_cast<uintptr_t>(y) % 16 == 0 && ldy % 8 == 0 && offsets == nullptr &&
                     ceil_div(tokens, kTokens) * ceil_div(rows, kPairRows) * 2 > info->sm_count;
  if (y_tma && !make_tensor_map_2d(&ymap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y, rows, tokens, ldy * 2, 32, 32,
                                   CU_TENSOR_MAP_SWIZZLE_64B))
    return GPTQ_ERR_CUDA;
  auto run = [&](auto launch) { return launch(wmap, xmap, xwide, wsmap, xsmap, ymap, a, info, st); };
  if (y_tma)
    return nv ? run(launch_pair_of<true, __nv_bfloat16, kTokens, true>) : run(launch_pair_of<false, __nv_bfloat16, kTokens, true>);
  if (y_bf16) return nv ? run(launch_pair<true, __nv_bfloat16>) : run(launch_pair<false, __nv_bfloat16>);
  return nv ? run(launch_pair<true, float>) : run(launch_pair<false, float>);
}

}  // namespace gptq
