// Products of 4-bit floating-point matrices on the tensor cores, dense and
// grouped by expert:
//
//   y[i, r] = tw[g] tx[g] sum_c W[g, r, c] X[i, c],  i in group g's rows of X
//
// with both operands as E2M1 codes and block scales (fp4.cuh).  The block
// scales are multiplied in by the tensor cores (tcgen05.mma .block_scale), the
// sums are fp32, the tensor scales are multiplied in at the end.
//
// Roles are turned round against the usual: the 128 rows of an MMA are rows of
// W and its N columns are tokens, so that a single token is an MMA of N = 16
// and every group's last tile only as wide as its tokens, and 32 lanes of an
// accumulator column are 32 neighbouring outputs of one token.
//
// One CTA a tile of 128 weight rows x up to 256 tokens, persistent over the
// tiles; TMA brings 256 columns of K a stage (128 bytes a row, 128-byte
// swizzle), bulk copies bring the stage's scale tiles, tcgen05.cp takes those
// to tensor memory (each stage has its own columns there, so that no copy
// meets a product that still reads the last ones).
#include <algorithm>
#include <atomic>

#include "fp4.cuh"

namespace gptq {
namespace {

constexpr int kRows = 128;    // weight rows of a tile
constexpr int kTokens = 256;  // tokens of a tile at most
constexpr int kStageK = 256;  // columns of K a stage (128 bytes)
constexpr int kStages = 4;
constexpr int kBoxRows = 32;  // token rows a TMA box
constexpr int kABytes = kRows * kStageK / 2;
constexpr int kBBytes = kTokens * kStageK / 2;
constexpr int kSfBytes = kStageK / 64 * kFp4TileBytes;  // scales of 128 rows of a stage (nvfp4; half of it with mxfp4)
constexpr int kStageBytes = kABytes + kBBytes + 3 * kSfBytes;
constexpr int kThreads = 192;  // producer, MMA, 4 epilogue warps
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSfCol = 256, kSfStride = 64;  // scales of stage s at kSfCol + s * kSfStride: 16 columns of W's, 32 of X's
constexpr int kTableBytes = 3 * (kFp4MaxGroups + 1) * 4;
constexpr size_t kSmemBytes = 1024 + size_t(kStages) * kStageBytes + 256 + kTableBytes;
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
  int* status;
  uint64_t wait_ns;
};

// kind::mxf4nvf4 with a scale every 16 columns (E4M3), kind::mxf4 every 32 (2^e).
template <bool NV>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
  if (NV)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of the block-scaled kinds: E2M1 operands along K,
// scale type (0 E4M3, 1 2^e), M = 128, N tokens; `pair` picks the byte pair of
// the 32-bit scale cell (mxfp4 uses two bytes an MMA).
__device__ __forceinline__ uint32_t fp4_idesc(bool nv, uint32_t n, uint32_t pair) {
  return (pair * 2) << 4 | 1u << 7 | 1u << 10 | (n >> 3) << 17 | (nv ? 0u : 1u) << 23 | 1u << 27 | (pair * 2) << 29;
}

// A scale tile (512 bytes of shared memory, 32 rows of 16 bytes) to four
// tensor-memory columns, the same for each quarter of the lanes.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t smem) {
  const uint64_t desc = static_cast<uint64_t>((smem >> 4) & 0x3FFFu) | 8ull << 32 | 1ull << 46;  // 8 rows apart: 128 bytes
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

struct Tile {
  int g;
  int token;   // first token (row of X)
  int count;   // tokens of the tile
  int cols;    // MMA columns: count rounded up to 16
  int64_t xband;  // first band of X's scales
  int wtile;   // tile of W's rows in the group
};

template <bool NV, typename OUT>
__global__ void __launch_bounds__(kThreads, 1)
    fp4_matmul_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, MatmulArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + size_t(kStages) * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* drain = acc_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* table = reinterpret_cast<int*>(smem + size_t(kStages) * kStageBytes + 256);
  const GroupTable t{table, table + kFp4MaxGroups + 1, table + 2 * (kFp4MaxGroups + 1)};

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  constexpr int kBlk = NV ? 16 : 32;
  constexpr int kStageQuads = kStageK / (4 * kBlk);  // scale tiles of a stage along K
  constexpr int kQuadMmas = kBlk / 16;               // MMAs a scale tile serves

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 4);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&wmap);
    prefetch_tensormap(&xmap);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();
  pdl_wait();
  bool ok_groups = true;
  if (a.offsets != nullptr) {
    ok_groups = build_groups(t, a.offsets, a.groups, a.tokens, kTokens);
    if (!ok_groups && blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, GPTQ_ERR_INVALID_ARG);
  } else {
    if (threadIdx.x == 0) {
      t.off[0] = t.band[0] = t.tile[0] = 0;
      t.off[1] = static_cast<int>(a.tokens);
      t.band[1] = static_cast<int>((a.tokens + kFp4Band - 1) / kFp4Band);
      t.tile[1] = static_cast<int>((a.tokens + kTokens - 1) / kTokens);
    }
    __syncthreads();
  }
  const int wtiles = static_cast<int>((a.rows + kRows - 1) / kRows);
  const int64_t items = ok_groups ? static_cast<int64_t>(t.tile[a.groups]) * wtiles : 0;
  const int quads = fp4_quads(a.n, NV);
  const int mmas = (a.n + 63) / 64;
  const int kstages = (a.n + kStageK - 1) / kStageK;

  auto tile_of = [&](int64_t item) {
    Tile x;
    const int tt = static_cast<int>(item / wtiles);
    x.wtile = static_cast<int>(item - static_cast<int64_t>(tt) * wtiles);
    x.g = find_group(t.tile, a.groups, tt);
    const int j = tt - t.tile[x.g];
    x.token = t.off[x.g] + j * kTokens;
    x.count = min(kTokens, t.off[x.g + 1] - x.token);
    x.cols = (x.count + 15) / 16 * 16;
    x.xband = t.band[x.g] + j * (kTokens / kFp4Band);
    return x;
  };

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- producer ----------------
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_parity = 0;
      for (int64_t item = blockIdx.x; item < items && !*abort_flag; item += gridDim.x) {
        const Tile x = tile_of(item);
        const int boxes = (x.cols + kBoxRows - 1) / kBoxRows;
        const int halves = x.cols > kFp4Band ? 2 : 1;
        const int wy = static_cast<int>(x.g * a.rows) + x.wtile * kRows;
        const uint8_t* wsc = a.wscales + (static_cast<int64_t>(x.g) * wtiles + x.wtile) * quads * kFp4TileBytes;
        const uint8_t* xsc = a.xscales + x.xband * quads * kFp4TileBytes;
        for (int kb = 0; kb < kstages; ++kb) {
          if (!mbar_wait(empty + stage, phase ^ 1u, a.wait_ns)) {
            set_status(a.status, GPTQ_ERR_TIMEOUT);
            *abort_flag = 1;
            break;
          }
          if (*abort_flag) break;
          uint8_t* sa = smem + size_t(stage) * kStageBytes;
          uint8_t* sb = sa + kABytes;
          uint8_t* ssa = sb + kBBytes;
          uint8_t* ssb = ssa + kSfBytes;
          const uint32_t sf = static_cast<uint32_t>(min(kStageQuads, quads - kb * kStageQuads) * kFp4TileBytes);
          const int64_t sf_at = static_cast<int64_t>(kb) * kStageQuads * kFp4TileBytes;
          mbar_arrive_expect_tx(full + stage, kABytes + boxes * (kBoxRows * kStageK / 2) + (1 + halves) * sf);
          tma_load_2d(sa, &wmap, full + stage, kb * (kStageK / 2), wy);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(sb + b * (kBoxRows * kStageK / 2), &xmap, full + stage, kb * (kStageK / 2), x.token + b * kBoxRows);
          bulk_load(ssa, wsc + sf_at, sf, full + stage);
          for (int h = 0; h < halves; ++h)
            bulk_load(ssb + h * kSfBytes, xsc + h * static_cast<int64_t>(quads) * kFp4TileBytes + sf_at, sf, full + stage);
          issued |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every stage that was armed has received its bytes
      for (int s = 0; s < kStages; ++s)
        if (issued & (1u << s))
          if (!mbar_wait(full + s, (issued_parity >> s) & 1u, kDrainNs)) set_status(a.status, GPTQ_ERR_TIMEOUT);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- MMA issuer ----------------
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int64_t item = blockIdx.x; item < items && ok; item += gridDim.x, acc_phase ^= 1u) {
        const Tile x = tile_of(item);
        const int halves = x.cols > kFp4Band ? 2 : 1;
        if (!mbar_wait(acc_empty, acc_phase ^ 1u, a.wait_ns) || *abort_flag) {
          set_status(a.status, GPTQ_ERR_TIMEOUT);
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        for (int kb = 0; kb < kstages; ++kb) {
          if (!mbar_wait(full + stage, phase, a.wait_ns) || *abort_flag) {
            set_status(a.status, GPTQ_ERR_TIMEOUT);
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + size_t(stage) * kStageBytes);
          const uint32_t sb = sa + kABytes, ssa = sb + kBBytes, ssb = ssa + kSfBytes;
          const uint32_t tsa = tmem + kSfCol + stage * kSfStride, tsb = tsa + 16;
          const int q = min(kStageQuads, quads - kb * kStageQuads);
          for (int i = 0; i < q; ++i) {
            copy_scales(tsa + 4 * i, ssa + i * kFp4TileBytes);
            for (int h = 0; h < halves; ++h) copy_scales(tsb + 8 * i + 4 * h, ssb + h * kSfBytes + i * kFp4TileBytes);
          }
          const int m = min(kStageK / 64, mmas - kb * (kStageK / 64));
          for (int i = 0; i < m; ++i) {
            const int qi = i / kQuadMmas;
            mma_fp4<NV>(tmem, smem_desc_sw128(sa + 32 * i, 16, 1024), smem_desc_sw128(sb + 32 * i, 16, 1024),
                        fp4_idesc(NV, x.cols, i % kQuadMmas), tsa + 4 * qi, tsb + 8 * qi, kb > 0 || i > 0);
          }
          mma_commit(empty + stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit(acc_full);
      }
      mma_commit(drain);
      if (!mbar_wait(drain, 0u, kDrainNs)) set_status(a.status, GPTQ_ERR_TIMEOUT);
    }
  } else {
    // ---------------- epilogue ----------------
    const int quad = warp & 3;  // the tensor-memory lanes of this warp
    uint32_t acc_phase = 0;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x, acc_phase ^= 1u) {
      const Tile x = tile_of(item);
      int ok = 1;
      if (lane == 0) {
        ok = mbar_wait(acc_full, acc_phase, a.wait_ns) && !*abort_flag;
        if (!ok) {
          set_status(a.status, GPTQ_ERR_TIMEOUT);
          *abort_flag = 1;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const float tw = a.wt != nullptr ? a.wt[x.g] : 1.0f, tx = a.xt != nullptr ? a.xt[x.g] : 1.0f;
      const int64_t r = static_cast<int64_t>(x.wtile) * kRows + quad * 32 + lane;
      OUT* out = static_cast<OUT*>(a.y) + static_cast<int64_t>(x.token) * a.ldy + r;
      for (int c = 0; c < x.count; c += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(quad * 32) << 16) + c, v);
        tmem_ld_wait();
        if (r < a.rows) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + j < x.count) store_out(out + static_cast<int64_t>(c + j) * a.ldy, __uint_as_float(v[j]) * tw * tx);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <bool NV, typename OUT>
gptq_status launch_matmul(const CUtensorMap& wmap, const CUtensorMap& xmap, const MatmulArgs& a, int64_t items,
                          const DeviceInfo* info, cudaStream_t st) {
  static std::atomic<bool> attr_set[64] = {};  // per device, shared by host threads
  if (!attr_set[info->device]) {
    if (cudaFuncSetAttribute(fp4_matmul_kernel<NV, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemBytes)) != cudaSuccess)
      return GPTQ_ERR_CUDA;
    attr_set[info->device] = true;
  }
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(items, info->sm_count));
  if (launch_pdl(fp4_matmul_kernel<NV, OUT>, grid, kThreads, kSmemBytes, st, wmap, xmap, a) != cudaSuccess)
    return GPTQ_ERR_CUDA;
  return launch_status();
}

}  // namespace

gptq_status fp4_matmul(bool nv, const uint8_t* wq, const uint8_t* wscales, const float* wt, int groups, int64_t rows,
                       int n, const uint8_t* xq, const uint8_t* xscales, const float* xt, int64_t tokens,
                       const int32_t* offsets, void* y, int y_bf16, int64_t ldy, cudaStream_t st) {
  const DeviceInfo* info = device_info();
  if (info == nullptr) return GPTQ_ERR_CUDA;
  const int64_t pitch = fp4_pitch(n);
  CUtensorMap wmap, xmap;
  if (!make_tensor_map_2d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, wq, pitch, static_cast<uint64_t>(groups) * rows, pitch,
                          kStageK / 2, kRows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tensor_map_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, pitch, tokens, pitch, kStageK / 2, kBoxRows,
                          CU_TENSOR_MAP_SWIZZLE_128B))
    return GPTQ_ERR_CUDA;
  MatmulArgs a;
  a.wscales = wscales;
  a.xscales = xscales;
  a.wt = wt;
  a.xt = xt;
  a.offsets = offsets;
  a.groups = groups;
  a.rows = rows;
  a.tokens = tokens;
  a.n = n;
  a.y = y;
  a.ldy = ldy;
  a.status = info->status;
  a.wait_ns = wait_limit_ns();
  // token tiles: each group's last one may be part full
  const int64_t tiles = offsets == nullptr ? ceil_div(tokens, kTokens) : tokens / kTokens + std::min<int64_t>(groups, tokens);
  const int64_t items = tiles * ceil_div(rows, kRows);
  if (nv)
    return y_bf16 ? launch_matmul<true, __nv_bfloat16>(wmap, xmap, a, items, info, st)
                  : launch_matmul<true, float>(wmap, xmap, a, items, info, st);
  return y_bf16 ? launch_matmul<false, __nv_bfloat16>(wmap, xmap, a, items, info, st)
                : launch_matmul<false, float>(wmap, xmap, a, items, info, st);
}

}  // namespace gptq
