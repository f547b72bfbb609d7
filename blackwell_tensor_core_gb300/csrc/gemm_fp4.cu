// Products of microscaled 4-bit matrices on tcgen05 tensor cores (sm_103a):
//   D[i, n] = alpha sum_k A[i, k] B[n, k]
// with A the activations [M, K] and B the weights [N, K] (or one [N, K] per
// group of rows of A), both e2m1 with a scale per block of 16 or 32 columns
// (fp4.h), FP32 accumulation, alpha the product of the matrices' FP32 scales.
//
// The kernel computes D^T: 128 weight rows per CTA are the M of an
// instruction and the activations' rows its N, which may be any multiple of
// 16 up to 192.  So a ragged end of a group costs what it has rows, not a
// 256-row tile.  A CTA pair (cta_group::2) takes 256 or 512 weight rows x 192
// activation rows; each CTA stages its own weight rows and half of the
// activation rows.
//
// Scales travel as their 512-byte tiles: TMA brings them beside the operands
// and tcgen05.cp puts them into TMEM, four columns a tile, in order with the
// MMAs of the same thread.  Activation tiles start at multiples of 192 rows,
// so a tile's first scale row is a multiple of 64: the MMA reads the scales
// of its N from the TMEM column of that row's group of 32.
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <mutex>
#include <type_traits>

#include "../../include/bwgemm.h"
#include "fp4.h"
#include "launch.h"
#include "params.h"
#include "ptx.cuh"
#include "runtime.h"

namespace bwg {
namespace {

constexpr int kFp4MaxGroups = 1024;
constexpr int kTok = 192;          // activation rows of a tile: the MMA's N
constexpr int kKBytes = 128;       // one stage: 256 columns, one swizzle row
constexpr int kKCols = 256;
constexpr uint32_t kWBytes = 128 * kKBytes;        // a CTA's weight rows of one consumer
constexpr uint32_t kTokBytes = (kTok / 2) * kKBytes;  // a CTA's half of the activation rows

struct Fp4GemmParams {
  CUtensorMap map_w;   // weights {K/2 bytes, N, G}, box {128, 128, 1}, 128B swizzle
  CUtensorMap map_a;   // activations {K/2 bytes, M}, box {128, 96}, 128B swizzle
  CUtensorMap map_ws;  // weight scales {128 words, K tiles, row blocks}, box {128, 4 or 2, 1}
  CUtensorMap map_as;  // activation scales, the same with a box of 2 row blocks
  unsigned long long* err;
  unsigned long long timeout_ns;
  uint32_t tx_extra;       // test hook: extra bytes expected per stage (0 normally)
  const int* offsets;      // [G + 1] or nullptr: one group of all M rows
  const float* a_global;   // nullptr: 1
  const float* b_global;   // nullptr: 1
  void* d;
  long long ldd;
  int M, N, G;             // N: output columns (SwiGLU: half of the weights' rows)
  int b_globals;           // 1 or G
  int num_k_blocks, last_steps;  // stages, and 64-column steps of the last one
  int num_w_tiles;         // tiles along the weights
  int w_blocks;            // scale row blocks of one group's weights
  int swiglu_up;           // SwiGLU: first weight row of the up half
  int out_dtype, group_m;
};

enum : uint32_t { kRoleProducer = 0, kRoleMma = 1, kRoleEpilogue = 2 };
enum : uint32_t { kBarFull = 0, kBarEmpty = 1, kBarAccFull = 2, kBarAccEmpty = 3 };

__device__ __forceinline__ void record_fault(unsigned long long* err, unsigned long long kind, uint32_t role,
                                             uint32_t bar, uint32_t stage, uint32_t phase) {
  const unsigned long long code = (kind << 56) | (static_cast<unsigned long long>(role) << 48) |
                                  (static_cast<unsigned long long>(bar) << 40) |
                                  (static_cast<unsigned long long>(blockIdx.x & 0xFFFFFFu) << 16) |
                                  ((stage & 0xFFu) << 8) | (phase & 0xFFu);
  atomicCAS(err, 0ull, code);
}

// Group tables in shared memory: rows of each group (lo[g] .. lo[g + 1], from
// the offsets clamped into [0, M] and made non-decreasing), its first scale
// row and the tiles before it.  Built by one warp.
struct Tables {
  int* lo;      // [G + 1]
  int* prefix;  // [G + 1]
  int* sf;      // [G]
};

__device__ bool build_tables(const Fp4GemmParams& p, const Tables& t) {
  const int lane = static_cast<int>(threadIdx.x & 31u);
  int run = 0, carry_t = 0, carry_s = 0;
  bool bad = false;
  for (int g0 = 0; g0 < p.G; g0 += 32) {
    const int g = g0 + lane;
    const bool in = g < p.G;
    const int a = !in ? 0 : p.offsets != nullptr ? p.offsets[g] : 0;
    const int b = !in ? 0 : p.offsets != nullptr ? p.offsets[g + 1] : p.M;
    if (in && ((g == 0 && a != 0) || b < a || a < 0 || b > p.M)) bad = true;
    int m = in ? max(a, b) : run;
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, m, d);
      if (lane >= d) m = max(m, y);
    }
    const int hi = min(max(m, run), p.M);
    int lo = __shfl_up_sync(0xffffffffu, hi, 1);
    if (lane == 0) lo = run;
    const int rows = in ? hi - lo : 0;
    const int tiles = (rows + kTok - 1) / kTok * p.num_w_tiles;
    int it = tiles, is = pad128(rows);
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, it, d);
      const int z = __shfl_up_sync(0xffffffffu, is, d);
      if (lane >= d) {
        it += y;
        is += z;
      }
    }
    if (in) {
      t.lo[g] = lo;
      t.lo[g + 1] = hi;
      t.prefix[g] = carry_t + it - tiles;
      t.prefix[g + 1] = carry_t + it;
      t.sf[g] = carry_s + is - pad128(rows);
    }
    carry_t += __shfl_sync(0xffffffffu, it, 31);
    carry_s += __shfl_sync(0xffffffffu, is, 31);
    run = __shfl_sync(0xffffffffu, hi, 31);
    __syncwarp();
  }
  return !__any_sync(0xffffffffu, bad);
}

struct Tile {
  int g;
  int w0;       // first weight row (of the gate half for SwiGLU)
  int t0;       // first activation row
  int tokens;   // rows, 1 .. kTok
  int n;        // tokens rounded up to 16
  int srow;     // scale row of t0 in the activation scales
};

template <int W_ROWS>
__device__ __forceinline__ Tile tile_at(const Fp4GemmParams& p, const Tables& t, int u) {
  int g = 0, top = p.G - 1;
  while (g < top) {
    const int mid = (g + top + 1) >> 1;
    if (t.prefix[mid] <= u)
      g = mid;
    else
      top = mid - 1;
  }
  const int rows = t.lo[g + 1] - t.lo[g];
  int tt, wt;
  raster_tile(u - t.prefix[g], (rows + kTok - 1) / kTok, p.num_w_tiles, p.group_m, &tt, &wt);
  Tile r;
  r.g = g;
  r.w0 = wt * W_ROWS;
  r.t0 = t.lo[g] + tt * kTok;
  r.tokens = min(kTok, rows - tt * kTok);
  r.n = (r.tokens + 15) & ~15;
  r.srow = t.sf[g] + tt * kTok;
  return r;
}

// The tiles of one cluster, u = first, first + stride, .., looked up 32 at a
// time, a lane each: the divisions and the group search of a tile switch
// then cost a warp once in 32 tiles.
template <int W_ROWS>
struct TileWindow {
  const Fp4GemmParams& p;
  const Tables& tb;
  int first, stride, count;
  int base;  // tile of lane 0, -1 before the first
  Tile mine;

  __device__ TileWindow(const Fp4GemmParams& p_, const Tables& tb_, int first_, int stride_, int total)
      : p(p_), tb(tb_), first(first_), stride(stride_), base(-32) {
    count = first < total ? (total - first + stride - 1) / stride : 0;
  }
  __device__ bool have(int i) const { return i < count; }
  __device__ void seek(int i) {
    if (i - base < 32) return;
    base = i;
    const int at = i + static_cast<int>(threadIdx.x & 31u);
    mine = tile_at<W_ROWS>(p, tb, first + (at < count ? at : i) * stride);
  }
  __device__ Tile at(int i) {
    seek(i);
    Tile t;
    t.g = __shfl_sync(0xffffffffu, mine.g, i - base);
    t.w0 = __shfl_sync(0xffffffffu, mine.w0, i - base);
    t.t0 = __shfl_sync(0xffffffffu, mine.t0, i - base);
    t.tokens = __shfl_sync(0xffffffffu, mine.tokens, i - base);
    t.srow = __shfl_sync(0xffffffffu, mine.srow, i - base);
    t.n = (t.tokens + 15) & ~15;
    return t;
  }
  // N and the column shift of the activation scales (n << 2 | shift), as a
  // value the compiler knows to be the same in every lane.
  __device__ uint32_t mma_values(int i) {
    seek(i);
    const bool me = static_cast<int>(threadIdx.x & 31u) == i - base;
    return __reduce_max_sync(0xffffffffu, me ? (static_cast<uint32_t>(mine.n) << 2) |
                                                   (static_cast<uint32_t>(mine.srow & 127) / 32u)
                                             : 0u);
  }
};

// A sum times the operands' scales: sum * pre * post.  pre is 1 where the scales'
// product is a normal FP32 number; else they are two factors, the larger one first
// if it is too small and the smaller one first if it is too large: sums are below
// 2^55 and no less than 2^-20, so that the first product then keeps its bits
// wherever the second is representable.  pre stands in a branch of its own
// (multiplying by it always: SwiGLU of 32768 rows 186 us instead of 180).
struct Alpha {
  float pre, post;
  template <int N>
  __device__ __forceinline__ void apply_pre(uint32_t (&v)[N]) const {
    if (pre != 1.f) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __float_as_uint(pre * __uint_as_float(v[i]));
    }
  }
  __device__ __forceinline__ float apply_post(uint32_t v) const { return post * __uint_as_float(v); }
};
__device__ __forceinline__ float scale_at(const float* p) { return p != nullptr ? *p : 1.f; }
__device__ __forceinline__ Alpha alpha_of(float x, float y) {
  const float p = x * y, size = fabsf(p);
  if (!(size < 1.17549435e-38f || size > 3.4028235e38f)) return {1.f, p};
  const bool swap = (fabsf(x) < fabsf(y)) == (size < 1.f);
  return swap ? Alpha{y, x} : Alpha{x, y};
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g * rcp_approx(1.0f + __expf(-g)) * u; }

// Warps 0, 2 and 3 load, warp 1 issues the MMAs, warps 4.. are the epilogue.
constexpr int kPairThreads = 384;
// Ring depth: the MMA loop is unrolled over it, so that every stage's
// addresses are constants.
constexpr int stages_of(int nc) { return nc == 1 ? 6 : 4; }

// Two blocks: registers per thread after set-up, out of 168 x 384 at launch.
constexpr uint32_t kRegsControl = 56, kRegsEpilogue = 224;
static_assert(kRegsControl * 128 + kRegsEpilogue * 256 <= 168 * 384, "the register split must fit");

// Shared memory: stage s holds [NC weight blocks][activation rows][scales].
template <int NC>
struct Layout {
  static constexpr uint32_t kScaleTiles = 4;  // K tiles of a stage with blocks of 16 (2 with blocks of 32)
  static constexpr uint32_t kStageW = NC * kWBytes;
  static constexpr uint32_t kSfBlock = kScaleTiles * kScaleTileBytes;  // scales of 128 rows of one stage
  static constexpr uint32_t kStageSf = (NC + 2) * kSfBlock;
  static constexpr uint32_t kStage = kStageW + kTokBytes + kStageSf;
  static_assert(kStage % 1024 == 0, "swizzled tiles start on 1024 bytes");
};

// NC weight blocks of 128 rows a CTA x up to 192 rows of A.  NC == 1: two
// accumulators, so that the epilogue of a tile runs beside the MMAs of the
// next.  NC == 2: one accumulator a block; fewer bytes staged and fewer
// instructions issued per tile, but the tensor cores idle about 1600 clocks at
// a tile's end.  SW: the two blocks are the gate and the up rows of the same
// 256 output columns.
// What bounds it: with random data the power limit (8192^3 NVFP4 160 us in a
// short run at 2070 MHz, 182 back to back at 1.87-1.95 GHz and 1370 W); at full
// clock the MMA warp's issue and the staging: a k-block of an NC == 2 tile
// takes 0.42 us (0.39 MXFP4) where its MMAs need 0.371, one of an NC == 1 tile
// 0.24 (0.21) for 0.186.
template <int NC, int FMT, bool SW>
__global__ void __launch_bounds__(kPairThreads, 1) fp4_pair_kernel(const __grid_constant__ Fp4GemmParams p) {
  static_assert(!SW || NC == 2, "SwiGLU pairs a gate block with an up block");
  using L = Layout<NC>;
  constexpr int kVec = FMT == kNvfp4 ? 16 : 32;
  constexpr int kTilesK = FMT == kNvfp4 ? 4 : 2;     // scale tiles of a stage along K
  constexpr uint32_t kSfBytes = kTilesK * kScaleTileBytes;
  constexpr uint32_t kStageTx = 2u * (L::kStageW + kTokBytes + (NC + 2) * kSfBytes);
  constexpr int kWRows = SW ? 256 : 256 * NC;        // output columns of a tile
  constexpr uint32_t kAccCols = kTok;
  constexpr uint32_t kSfCol0 = 2 * kTok;             // scales start after the two accumulators
  constexpr uint32_t kSfCols = (NC + 2) * kTilesK * 4;  // TMEM columns of one stage's scales
  static_assert(kSfCol0 + kSfCols <= kTmemCols, "two accumulators and a stage's scales");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t rank = cluster_ctarank();
  constexpr int S = stages_of(NC);
  const uint32_t bars = base + static_cast<uint32_t>(S) * L::kStage;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
  auto acc_full = [&](int a) { return bars + 8u * (2 * S + a); };
  auto acc_empty = [&](int a) { return bars + 8u * (2 * S + 2 + a); };
  const uint32_t tmem_slot = bars + 8u * (2 * S + 4);
  int* tab = reinterpret_cast<int*>(smem_raw + (tmem_slot + 16u - smem_u32(smem_raw)));
  const Tables tb{tab, tab + p.G + 1, tab + 2 * p.G + 2};

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(acc_full(a), 1);
      // epilogue warps of both CTAs that read this accumulator
      mbar_init(acc_empty(a), NC == 1 || SW ? 16 : 8);
    }
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&p.map_w);
    prefetch_tensormap(&p.map_a);
    prefetch_tensormap(&p.map_ws);
    prefetch_tensormap(&p.map_as);
  }
  if (warp == 1) {
    tmem_alloc<2>(tmem_slot, kTmemCols);
    tmem_relinquish<2>();
  }
  grid_dependency_wait();
  if (warp == 4) {
    const bool ok = build_tables(p, tb);
    if (!ok && blockIdx.x == 0 && lane == 0) record_fault(p.err, kFaultBadOffsets, 0, 0, 0, 0);
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const int first = static_cast<int>(cluster_id_x());
  const int stride = static_cast<int>(num_clusters_x());
  const int total = tb.prefix[p.G];
  bool aborted = false;

  if (warp < 4) {
    // the epilogue warpgroups hold whole slices of accumulators
    if constexpr (NC == 2) setmaxnreg_dec<kRegsControl>();
    if (warp != 1) {
      // ---- TMA producers --------------------------------------------------------
      // One warp for each weight block and one for the activations.  A stage of
      // two blocks takes 6 loads; one diverged thread needs about 900 clocks to
      // issue them, more than the stage's MMAs (768).  Warps that stay together
      // and elect a lane need about 50 clocks a load, and three share them.
      const int job = warp == 0 ? 0 : static_cast<int>(warp) - 1;  // 0, 1: weight block, 2: activations
      if (job == 2 || job < NC) {
        int s = 0;
        uint32_t ph = 0;
        TileWindow<kWRows> win(p, tb, first, stride, total);
        for (int i = 0; win.have(i) && !aborted; ++i) {
          const Tile tl = win.at(i);
          const int row = job == 2 ? tl.t0 + static_cast<int>(rank) * (tl.n / 2)
                                   : tl.w0 + static_cast<int>(rank) * 128 + job * (SW ? p.swiglu_up : 256);
          const int sf_row = job == 2 ? tl.srow / 128 : tl.g * p.w_blocks + row / 128;
          for (int kb = 0; kb < p.num_k_blocks; ++kb) {
            if (!warp_wait_cta(empty_bar(s), ph ^ 1u, p.timeout_ns)) {
              if (lane == 0) record_fault(p.err, kFaultTimeout, kRoleProducer, kBarEmpty, s, ph ^ 1u);
              aborted = true;
              break;
            }
            if (elect_one()) {
              const uint32_t st = base + static_cast<uint32_t>(s) * L::kStage;
              const uint32_t fb = mapa_shared(full_bar(s), 0);
              if (job == 2) {
                tma_load_2d_pair(st + L::kStageW, &p.map_a, fb, kb * kKBytes, row);
                // both CTAs need the scales of all of the instruction's N; a
                // box of two row blocks (the second may lie past the end: zeros)
                tma_load_3d_pair(st + L::kStageW + kTokBytes + NC * L::kSfBlock, &p.map_as, fb, 0, kb * kTilesK, sf_row);
              } else {
                if (job == 0 && rank == 0) mbar_arrive_expect_tx(full_bar(s), kStageTx + p.tx_extra);
                tma_load_3d_pair(st + job * kWBytes, &p.map_w, fb, kb * kKBytes, row, tl.g);
                tma_load_3d_pair(st + L::kStageW + kTokBytes + job * L::kSfBlock, &p.map_ws, fb, 0, kb * kTilesK, sf_row);
              }
            }
            __syncwarp();
            if (++s == S) {
              s = 0;
              ph ^= 1u;
            }
          }
        }
      }
    } else {
      // ---- MMA issuer (CTA 0 of the pair) ------------------------------------
      // A stage is 10 to 24 tcgen05 instructions, and their issue, not the
      // tensor cores, can set the pace.  So the operands are kept uniform (the
      // ring unrolled, tile values through a warp reduction, TMEM addresses
      // constant: all 512 columns are allocated, so they start at 0; the
      // operations predicated instead of issued in a branch), and a stage's
      // full barrier is asked before the stage before it is issued.
      if (rank == 0) {
        int s = 0, acc = 0;
        uint32_t ph = 0, acc_ph = 0;
        bool ready = false;
        TileWindow<kWRows> win(p, tb, first, stride, total);
        for (int i = 0; win.have(i) && !aborted; ++i) {
          const uint32_t packed = win.mma_values(i);
          const uint32_t shift = packed & 3u;
          const uint32_t idesc0 = make_idesc_fp4(FMT, 256, packed >> 2, 0);
          for (int a = 0; a < NC; ++a) {
            const int slot = NC == 1 ? acc : a;
            if (!warp_wait_all(acc_empty(slot), acc_ph ^ 1u, p.timeout_ns)) {
              if (lane == 0) record_fault(p.err, kFaultTimeout, kRoleMma, kBarAccEmpty, slot, acc_ph ^ 1u);
              aborted = true;
            }
          }
          if (aborted) break;
          tc_fence_after();
          int kb = 0;
          // one k-block, in stage st; returns false after the tile's last
          auto k_block = [&](auto stage_c) {
            constexpr int st = decltype(stage_c)::value;
            if (!ready && !warp_wait_cta(full_bar(st), ph, p.timeout_ns)) {
              if (lane == 0) record_fault(p.err, kFaultTimeout, kRoleMma, kBarFull, st, ph);
              aborted = true;
              return false;
            }
            tc_fence_after();
            constexpr int next = st + 1 == S ? 0 : st + 1;
            const bool ask = mbar_test_wait_cta(full_bar(next), next == 0 ? ph ^ 1u : ph);
            uint32_t mem = base + static_cast<uint32_t>(st) * L::kStage;
            // the stage's descriptors are computed here, not kept in registers
            // for all stages (80 registers instead of 120, and no spills with
            // the SwiGLU kernel's register split)
            asm volatile("" : "+r"(mem));
            const uint32_t sf = mem + L::kStageW + kTokBytes;
            const int steps = kb + 1 == p.num_k_blocks ? p.last_steps : 4;
            const bool on = elect_one();
            // scales: block c's tile j to columns (c * kTilesK + j) * 4, the
            // activations' two row blocks of tile j side by side
#pragma unroll
            for (int j = 0; j < kTilesK; ++j) {
#pragma unroll
              for (int c = 0; c < NC; ++c)
                tmem_copy_scales_if<2>(on, kSfCol0 + (c * kTilesK + j) * 4,
                                      make_smem_desc(sf + c * L::kSfBlock + j * kScaleTileBytes, 16, 128, kSwizzleNone));
              const uint32_t sfb = sf + NC * L::kSfBlock + j * kScaleTileBytes;
              constexpr uint32_t kSfb = kSfCol0 + NC * kTilesK * 4;
              tmem_copy_scales_if<2>(on, kSfb + 8 * j, make_smem_desc(sfb, 16, 128, kSwizzleNone));
              tmem_copy_scales_if<2>(on, kSfb + 8 * j + 4, make_smem_desc(sfb + kSfBytes, 16, 128, kSwizzleNone));
            }
            const uint64_t b_desc = make_smem_desc(mem + L::kStageW, 16, 1024, kSwizzle128B);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const int j = FMT == kNvfp4 ? kk : kk / 2;
              const uint32_t idesc = FMT == kNvfp4 ? idesc0
                                                   : (idesc0 | (static_cast<uint32_t>(kk & 1) << 5) |
                                                      (static_cast<uint32_t>(kk & 1) << 30));
#pragma unroll
              for (int c = 0; c < NC; ++c) {
                const uint64_t a_desc = make_smem_desc(mem + static_cast<uint32_t>(c) * kWBytes, 16, 1024, kSwizzle128B);
                mma_fp4_if<2, kVec>(on && kk < steps, static_cast<uint32_t>(NC == 1 ? acc : c) * kAccCols, a_desc + kk * 2,
                                   b_desc + kk * 2, idesc, kSfCol0 + (c * kTilesK + j) * 4,
                                   kSfCol0 + (NC * kTilesK + 2 * j) * 4 + shift, (kb | kk) != 0 ? 1u : 0u);
              }
            }
            mma_commit_pair_mc_if(on, empty_bar(st), 0x3);
            ready = __all_sync(0xffffffffu, ask);
            s = next;
            if (next == 0) ph ^= 1u;
            return ++kb < p.num_k_blocks;
          };
          while (true) {
            if (s == 0 && !k_block(std::integral_constant<int, 0>{})) break;
            if (s == 1 && !k_block(std::integral_constant<int, 1>{})) break;
            if (s == 2 && !k_block(std::integral_constant<int, 2>{})) break;
            if (s == 3 && !k_block(std::integral_constant<int, 3>{})) break;
            if constexpr (S > 4) {
              if (s == 4 && !k_block(std::integral_constant<int, 4>{})) break;
              if (s == 5 && !k_block(std::integral_constant<int, 5>{})) break;
            }
          }
          if (aborted) break;
          const bool on = elect_one();
          mma_commit_pair_mc_if(on, acc_full(NC == 1 ? acc : 0), 0x3);
          if (NC == 2) mma_commit_pair_mc_if(on, acc_full(1), 0x3);
          if constexpr (NC == 1) {
            acc ^= 1;
            if (acc == 0) acc_ph ^= 1u;
          } else {
            acc_ph ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else {
    if constexpr (NC == 2) setmaxnreg_inc<kRegsEpilogue>();
    // ---- epilogue: TMEM lane = output column, TMEM column = row of D --------
    const uint32_t q = warp & 3u;
    const int grp = static_cast<int>((warp - 4u) >> 2);  // SwiGLU: warpgroup 0 or 1
    const uint32_t acc_empty0 = mapa_shared(acc_empty(0), 0);
    const bool out32 = p.out_dtype == kOutF32;
    const bool outbf = p.out_dtype == kOutBF16;
    const uint32_t t_lane = (q * 32u) << 16;
    auto wait_acc_full = [&](int slot, uint32_t phase) {
      if (warp_wait_all(acc_full(slot), phase, p.timeout_ns)) return true;
      if (lane == 0) record_fault(p.err, kFaultTimeout, kRoleEpilogue, kBarAccFull, slot, phase);
      return false;
    };
    auto release = [&](int slot) {
      if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty0 + 8u * slot);
    };
    const float ga = scale_at(p.a_global);
    auto alpha_at = [&](int g) {
      return alpha_of(ga, p.b_global != nullptr ? p.b_global[p.b_globals > 1 ? g : 0] : 1.f);
    };
    // values of rows c0 .. c0 + 31 of the tile, this lane's column: 32 lanes
    // write 32 adjacent columns of one row at a time
    auto store = [&](const Tile& tl, int c0, const uint32_t (&v)[32]) {
      const int rows = tl.tokens - c0;
      const int col = tl.w0 + (NC == 2 && !SW ? grp * 256 : 0) + static_cast<int>(rank * 128u + q * 32u + lane);
      if (col >= p.N || rows <= 0) return;
      const int elt = out32 ? 4 : 2;
      const long long row_bytes = p.ldd * elt;
      uint8_t* dst = static_cast<uint8_t*>(p.d) + (static_cast<long long>(tl.t0 + c0) * p.ldd + col) * elt;
      if (out32) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (j < rows) *reinterpret_cast<uint32_t*>(dst) = v[j];
          dst += row_bytes;
        }
        return;
      }
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const float lo = __uint_as_float(v[j]), hi = __uint_as_float(v[j + 1]);
        const uint32_t pk = outbf ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
        if (j < rows) *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(pk);
        if (j + 1 < rows) *reinterpret_cast<uint16_t*>(dst + row_bytes) = static_cast<uint16_t>(pk >> 16);
        dst += 2 * row_bytes;
      }
    };
    TileWindow<kWRows> win(p, tb, first, stride, total);
    if constexpr (SW) {
      // The two warpgroups take alternate chunks of 32 rows, three each.  All
      // of a warp's gate and up values (192 registers) are read and both
      // accumulators handed back before the first silu: its exponentials
      // would hold the accumulators for about 2000 clocks longer.  Chunks past
      // the tile's rows end there (8 pairs of 4096 x 4096 18.2 -> 17.4 us, of
      // 512 x 512 7.4 -> 6.3).
      uint32_t acc_ph = 0;
      for (int i = 0; win.have(i); ++i) {
        if (!wait_acc_full(0, acc_ph) || !wait_acc_full(1, acc_ph)) {
          aborted = true;
          break;
        }
        acc_ph ^= 1u;
        tc_fence_after();
        const uint32_t col0 = t_lane + static_cast<uint32_t>(grp) * 32u;
        uint32_t gate[3][32], up[3][32];
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          // columns past the tile's rows lie inside the accumulators
          tmem_ld_32x32b_x32(col0 + c * 64, gate[c]);
          tmem_ld_32x32b_x32(col0 + kAccCols + c * 64, up[c]);
        }
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        release(0);
        release(1);
        const Tile tl = win.at(i);
        const Alpha alpha = alpha_at(tl.g);
        if (alpha.pre != 1.f) {
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            alpha.apply_pre(gate[c]);
            alpha.apply_pre(up[c]);
          }
        }
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          if (grp * 32 + c * 64 >= tl.tokens) break;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            gate[c][j] = __float_as_uint(silu_mul(alpha.apply_post(gate[c][j]), alpha.apply_post(up[c][j])));
          store(tl, grp * 32 + c * 64, gate[c]);
        }
      }
    } else if constexpr (NC == 2) {
      // each warpgroup its block's accumulator, all of it before the hand-back
      uint32_t acc_ph = 0;
      for (int i = 0; win.have(i); ++i) {
        if (!wait_acc_full(grp, acc_ph)) {
          aborted = true;
          break;
        }
        acc_ph ^= 1u;
        tc_fence_after();
        uint32_t v[6][32];
#pragma unroll
        for (int c = 0; c < 6; ++c) tmem_ld_32x32b_x32(t_lane + static_cast<uint32_t>(grp) * kAccCols + c * 32, v[c]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        release(grp);
        const Tile tl = win.at(i);
        const Alpha alpha = alpha_at(tl.g);
#pragma unroll
        for (int c = 0; c < 6; ++c) {
          if (c * 32 >= tl.tokens) break;
          alpha.apply_pre(v[c]);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[c][j] = __float_as_uint(alpha.apply_post(v[c][j]));
          store(tl, c * 32, v[c]);
        }
      }
    } else {
      int acc = 0;
      uint32_t acc_ph = 0;
      for (int i = 0; win.have(i); ++i) {
        const Tile tl = win.at(i);
        const Alpha alpha = alpha_at(tl.g);
        if (!wait_acc_full(acc, acc_ph)) {
          aborted = true;
          break;
        }
        tc_fence_after();
        // the two warpgroups take alternate chunks of 32 rows (1900 rows of
        // 4096 x 1024 10.3 us, 11.5 with one)
        for (int c0 = grp * 32; c0 < tl.tokens; c0 += 64) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(t_lane + static_cast<uint32_t>(acc) * kAccCols + c0, v);
          tmem_wait_ld();
          if (c0 + 64 >= tl.tokens) {
            tc_fence_before();
            __syncwarp();
            release(acc);
          }
          alpha.apply_pre(v);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(alpha.apply_post(v[j]));
          store(tl, c0, v);
        }
        if (grp * 32 >= tl.tokens) release(acc);
        acc ^= 1;
        if (acc == 0) acc_ph ^= 1u;
      }
    }
    __syncwarp();
  }

  // ---- teardown -------------------------------------------------------------
  grid_dependents_launch();
  if (__syncthreads_or(aborted ? 1 : 0)) {
    // a wait gave up: let copies in flight land before their memory goes
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) nanosleep_ns(1000);
  }
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<2>(0, kTmemCols);
  }
}

// ---------------------------------------------------------- few rows -------
// At most 128 rows of A, where the weights' bytes are the time, and more where
// few rounds of its tiles cover them.  One CTA a tile of 128 output columns and
// up to 128 rows (rounded up to 16) as N.  Where there are too few tiles to
// keep the memory busy, a cluster of `split` CTAs shares a tile's k-blocks and
// sums its FP32 partials through distributed shared memory, in rank order;
// else the CTAs walk the tiles.
// What bounds it: HBM, and at a few MB of weights the latency of a launch and
// of the first loads (one row of 4096 x 4096 NVFP4 4.7 us, 128 rows 7.0, 256
// rows of 4096 x 7168 9.5).
constexpr int kSmallMaxRows = 128;
constexpr int kSmallThreads = 384;
// Threads of a launch: a second epilogue warpgroup where a tile has a second
// chunk of 32 rows (128 rows 0.3 us sooner, one row 0.15 later).
int small_threads(int rows) { return rows > 32 ? kSmallThreads : kSmallThreads - 128; }

constexpr int kSmallMaxStages = 8;
constexpr int kSmallMaxSplit = 8;

struct Fp4SmallParams {
  CUtensorMap map_w, map_a, map_ws, map_as;  // as above; activations in boxes of n rows, scales of one row block
  unsigned long long* err;
  unsigned long long timeout_ns;
  uint32_t tx_extra;       // test hook: extra bytes expected per stage (0 normally)
  const float* a_global;
  const float* b_global;
  void* d;
  long long ldd;
  int M, N, n;             // n: rows of a tile, a multiple of 16
  int num_k_blocks, last_steps;
  int tiles, split, stages, out_dtype;
  int row_tiles;           // tiles of up to 128 rows of A; a tile's number runs over them first
};

BWG_HD uint32_t small_stage_bytes(int n) {
  return kWBytes + static_cast<uint32_t>(n) * kKBytes + 2u * 4u * kScaleTileBytes;
}

// Four FP32 values of a CTA's shared memory in the cluster.
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

// Rank `rank` of p.split sums rows rank, rank + p.split, .. of a tile's partials
// (at `base` in each CTA, 128 floats a row), a warp a row, in rank order, and
// stores them.  All of a row's loads of 16 bytes are in flight; two rows at a
// time, or code for each cluster size, measured the same, 4 bytes a lane 0.3
// (16 rows) to 3 us more (128 rows).
__device__ __forceinline__ void sum_partials(const Fp4SmallParams& p, uint32_t base, int rank, int row0, int rows,
                                             int col0) {
  const bool out32 = p.out_dtype == kOutF32, outbf = p.out_dtype == kOutBF16;
  const Alpha alpha = alpha_of(scale_at(p.a_global), scale_at(p.b_global));
  const int ch = static_cast<int>(threadIdx.x & 31u) * 4;
  const int col = col0 + ch;
  const int elt = out32 ? 4 : 2;
  const bool whole =
      col + 4 <= p.N && ((reinterpret_cast<uintptr_t>(p.d) | static_cast<uintptr_t>(p.ldd * elt)) & (4 * elt - 1)) == 0;
  const int split = p.split;
  for (int j = rank + split * static_cast<int>(threadIdx.x >> 5); j < rows; j += split * static_cast<int>(blockDim.x >> 5)) {
    const uint32_t at = base + static_cast<uint32_t>(j * 128 + ch) * 4u;
    float4 part[kSmallMaxSplit];
#pragma unroll
    for (int c = 0; c < kSmallMaxSplit; ++c)
      if (c < split) part[c] = ld_cluster_v4(mapa_shared(at, static_cast<uint32_t>(c)));
    float x[4] = {part[0].x, part[0].y, part[0].z, part[0].w};
#pragma unroll
    for (int c = 1; c < kSmallMaxSplit; ++c)
      if (c < split) {
        x[0] += part[c].x;
        x[1] += part[c].y;
        x[2] += part[c].z;
        x[3] += part[c].w;
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = x[i] * alpha.pre * alpha.post;
    uint8_t* dst = static_cast<uint8_t*>(p.d) + (static_cast<long long>(row0 + j) * p.ldd + col) * elt;
    if (whole) {
      if (out32)
        *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
      else if (outbf)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
      else
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_f16x2(x[0], x[1]), pack_f16x2(x[2], x[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < p.N) {
          if (out32)
            reinterpret_cast<float*>(dst)[i] = x[i];
          else
            reinterpret_cast<uint16_t*>(dst)[i] = outbf ? cvt_rn_bf16(x[i]) : cvt_rn_f16(x[i]);
        }
    }
  }
}

// Column tile, first row and rows of tile t.  MANY: more than one row tile; its
// division would stand before the first loads of a call that has one (0.2 us of
// the 2.6 of 512 x 512, with what follows from it).
template <bool MANY>
struct SmallTile {
  int c, row0, rows;
  __device__ SmallTile(const Fp4SmallParams& p, int t) : c(t), row0(0), rows(p.M) {
    if constexpr (MANY) {
      c = t / p.row_tiles;
      row0 = (t - c * p.row_tiles) * kSmallMaxRows;
      rows = min(kSmallMaxRows, p.M - row0);
    }
  }
};

template <int FMT, bool MANY>
__global__ void __launch_bounds__(kSmallThreads, 1) fp4_small_kernel(const __grid_constant__ Fp4SmallParams p) {
  constexpr int kVec = FMT == kNvfp4 ? 16 : 32;
  constexpr int kTilesK = FMT == kNvfp4 ? 4 : 2;
  constexpr uint32_t kSfSlot = 4 * kScaleTileBytes;
  constexpr uint32_t kSfBytes = kTilesK * kScaleTileBytes;
  constexpr uint32_t kAcc = kSmallMaxRows;       // columns of one of two accumulators
  constexpr uint32_t kSfCol0 = 2 * kAcc;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31u;
  const int S = p.stages;
  const uint32_t stage_bytes = small_stage_bytes(p.n);
  const uint32_t a_bytes = static_cast<uint32_t>(p.n) * kKBytes;
  const uint32_t bars = base + static_cast<uint32_t>(S) * stage_bytes;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
  auto acc_full = [&](int a) { return bars + 8u * (2 * S + a); };
  auto acc_empty = [&](int a) { return bars + 8u * (2 * S + 2 + a); };
  const uint32_t tmem_slot = bars + 8u * (2 * S + 4);
  const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = p.split > 1 ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int stride = p.split > 1 ? p.tiles : static_cast<int>(gridDim.x);  // a cluster has one tile
  const int kb0 = p.num_k_blocks * rank / p.split, kb1 = p.num_k_blocks * (rank + 1) / p.split;
  bool aborted = false;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(acc_full(a), 1);
      mbar_init(acc_empty(a), (blockDim.x >> 5) - 4);
    }
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&p.map_w);
    prefetch_tensormap(&p.map_a);
    prefetch_tensormap(&p.map_ws);
    prefetch_tensormap(&p.map_as);
  }
  if (warp == 1) {
    tmem_alloc<1>(tmem_slot, kTmemCols);  // all columns: they start at 0
    tmem_relinquish<1>();
  }
  grid_dependency_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp == 0 || warp == 2) {
    // ---- TMA producers: weights, activations ---------------------------------
    const bool weights = warp == 0;
    const uint64_t policy = MANY ? l2_policy_evict_normal() : l2_policy_evict_first();
    int s = 0;
    uint32_t ph = 0;
    for (int t = first; t < p.tiles && !aborted; t += stride) {
      const SmallTile<MANY> tile(p, t);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!warp_wait_cta(empty_bar(s), ph ^ 1u, p.timeout_ns)) {
          if (lane == 0) record_fault(p.err, kFaultTimeout, kRoleProducer, kBarEmpty, s, ph ^ 1u);
          aborted = true;
          break;
        }
        if (elect_one()) {
          const uint32_t st = base + static_cast<uint32_t>(s) * stage_bytes;
          const uint32_t sf = st + kWBytes + a_bytes;
          if (weights) {
            mbar_arrive_expect_tx(full_bar(s), kWBytes + a_bytes + 2u * kSfBytes + p.tx_extra);
            tma_load_3d_hint(st, &p.map_w, full_bar(s), kb * kKBytes, tile.c * 128, 0, policy);
            tma_load_3d_hint(sf, &p.map_ws, full_bar(s), 0, kb * kTilesK, tile.c, policy);
          } else {
            tma_load_2d(st + kWBytes, &p.map_a, full_bar(s), kb * kKBytes, tile.row0);
            tma_load_3d(sf + kSfSlot, &p.map_as, full_bar(s), 0, kb * kTilesK, tile.row0 / 128);
          }
        }
        __syncwarp();
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer ------------------------------------------------------------
    int s = 0, acc = 0;
    uint32_t ph = 0, acc_ph = 0;
    const uint32_t idesc0 = make_idesc_fp4(FMT, 128, static_cast<uint32_t>(p.n), 0);
    for (int t = first; t < p.tiles && !aborted; t += stride) {
      if (!warp_wait_all(acc_empty(acc), acc_ph ^ 1u, p.timeout_ns)) {
        if (lane == 0) record_fault(p.err, kFaultTimeout, kRoleMma, kBarAccEmpty, acc, acc_ph ^ 1u);
        aborted = true;
        break;
      }
      tc_fence_after();
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!warp_wait_cta(full_bar(s), ph, p.timeout_ns)) {
          if (lane == 0) record_fault(p.err, kFaultTimeout, kRoleMma, kBarFull, s, ph);
          aborted = true;
          break;
        }
        tc_fence_after();
        const uint32_t st = base + static_cast<uint32_t>(s) * stage_bytes;
        const uint32_t sf = st + kWBytes + a_bytes;
        const int steps = kb + 1 == p.num_k_blocks ? p.last_steps : 4;
        const bool on = elect_one();
#pragma unroll
        for (int j = 0; j < kTilesK; ++j) {
          tmem_copy_scales_if<1>(on, kSfCol0 + j * 4,
                                 make_smem_desc(sf + j * kScaleTileBytes, 16, 128, kSwizzleNone));
          tmem_copy_scales_if<1>(on, kSfCol0 + (kTilesK + j) * 4,
                                 make_smem_desc(sf + kSfSlot + j * kScaleTileBytes, 16, 128, kSwizzleNone));
        }
        const uint64_t a_desc = make_smem_desc(st, 16, 1024, kSwizzle128B);
        const uint64_t b_desc = make_smem_desc(st + kWBytes, 16, 1024, kSwizzle128B);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const int j = FMT == kNvfp4 ? kk : kk / 2;
          const uint32_t idesc = FMT == kNvfp4 ? idesc0
                                               : (idesc0 | (static_cast<uint32_t>(kk & 1) << 5) |
                                                  (static_cast<uint32_t>(kk & 1) << 30));
          mma_fp4_if<1, kVec>(on && kk < steps, static_cast<uint32_t>(acc) * kAcc, a_desc + kk * 2, b_desc + kk * 2,
                              idesc, kSfCol0 + j * 4, kSfCol0 + (kTilesK + j) * 4, kb != kb0 || kk != 0 ? 1u : 0u);
        }
        mma_commit_1cta_if(on, empty_bar(s));
        if (kb + 1 == kb1) mma_commit_1cta_if(on, acc_full(acc));
        __syncwarp();
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
      acc ^= 1;
      if (acc == 0) acc_ph ^= 1u;
    }
  } else if (warp >= 4) {
    // ---- epilogue: TMEM lane = output column, TMEM column = row of D ---------
    const uint32_t q = warp & 3u;
    const bool out32 = p.out_dtype == kOutF32, outbf = p.out_dtype == kOutBF16;
    const Alpha alpha = alpha_of(scale_at(p.a_global), scale_at(p.b_global));
    int acc = 0;
    uint32_t acc_ph = 0;
    for (int t = first; t < p.tiles; t += stride) {
      if (!warp_wait_all(acc_full(acc), acc_ph, p.timeout_ns)) {
        if (lane == 0) record_fault(p.err, kFaultTimeout, kRoleEpilogue, kBarAccFull, acc, acc_ph);
        aborted = true;
        break;
      }
      tc_fence_after();
      const int ch = static_cast<int>(q * 32u + lane);
      const SmallTile<MANY> tile(p, t);
      const int col = tile.c * 128 + ch, row0 = tile.row0, rows = tile.rows;
      // the warpgroups take alternate chunks of 32 rows
      const int c_first = static_cast<int>((warp - 4u) >> 2) * 32, c_step = (static_cast<int>(blockDim.x >> 7) - 1) * 32;
      if (c_first >= rows && lane == 0) mbar_arrive_local(acc_empty(acc));
      for (int c0 = c_first; c0 < rows; c0 += c_step) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(((q * 32u) << 16) + static_cast<uint32_t>(acc) * kAcc + c0, v);
        tmem_wait_ld();
        if (c0 + c_step >= rows) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_local(acc_empty(acc));
        }
        if (p.split > 1) {
          // the ring is idle: every load of this CTA has been used
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c0 + j < rows) st_shared_u32(base + static_cast<uint32_t>((c0 + j) * 128 + ch) * 4u, v[j]);
        } else if (col < p.N) {
          alpha.apply_pre(v);
          const int elt = out32 ? 4 : 2;
          uint8_t* dst = static_cast<uint8_t*>(p.d) + (static_cast<long long>(row0 + c0) * p.ldd + col) * elt;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (c0 + j < rows) {
              const float x = alpha.apply_post(v[j]);
              if (out32)
                *reinterpret_cast<float*>(dst) = x;
              else
                *reinterpret_cast<uint16_t*>(dst) = outbf ? cvt_rn_bf16(x) : cvt_rn_f16(x);
            }
            dst += p.ldd * elt;
          }
        }
      }
      acc ^= 1;
      if (acc == 0) acc_ph ^= 1u;
    }
  }
  __syncwarp();

  grid_dependents_launch();
  if (p.split > 1) {
    const SmallTile<MANY> tile(p, first);
    // ---- partials: rank r sums rows r, r + split, .. of the tile ---------------
    cluster_sync_all();
    sum_partials(p, base, rank, tile.row0, tile.rows, tile.c * 128);
  }
  if (__syncthreads_or(aborted ? 1 : 0)) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) nanosleep_ns(1000);
  }
  if (p.split > 1) cluster_sync_all();  // peers may still read this CTA's partials
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(0, kTmemCols);
  }
}

// Whether a row (the same in all of a block's threads) is one of a group's: the
// clamped tables give it one where any of the offsets lies above it.
__device__ __forceinline__ bool row_has_group(const int* offsets, int G, int row) {
  bool above = false;
  for (int i = static_cast<int>(threadIdx.x); i <= G; i += static_cast<int>(blockDim.x)) above |= offsets[i] > row;
  return __syncthreads_or(above) != 0;
}

// A grouped product over no columns: zeros in the groups' rows, a block a row.
// The first block checks the offsets as build_tables does.
__global__ void fp4_zero_rows_kernel(const int* offsets, int G, int M, uint8_t* d, size_t ld_bytes, size_t row_bytes,
                                     unsigned long long* err) {
  grid_dependency_wait();
  const int row = static_cast<int>(blockIdx.x);
  if (row == 0) {
    bool bad = false;
    for (int g = static_cast<int>(threadIdx.x); g < G; g += static_cast<int>(blockDim.x)) {
      const int a = offsets[g], b = offsets[g + 1];
      bad |= (g == 0 && a != 0) || b < a || a < 0 || b > M;
    }
    if (bad) record_fault(err, kFaultBadOffsets, 0, 0, 0, 0);
  }
  if (!row_has_group(offsets, G, row)) return;
  for (size_t i = threadIdx.x; i < row_bytes; i += blockDim.x) d[static_cast<size_t>(row) * ld_bytes + i] = 0;
}

// SwiGLU of FP32 rows [gate | up], for halves that the fused epilogue cannot
// pair (it needs both to start on a tile of scales): the groups' rows only.
template <class T>
__global__ void fp4_swiglu_kernel(const float* x, const int* offsets, int G, int n_out, long long ldd, T* h) {
  grid_dependency_wait();
  const int row = static_cast<int>(blockIdx.x);
  if (row >= offsets[G] && !row_has_group(offsets, G, row)) return;
  const float* r = x + static_cast<long long>(row) * 2 * n_out;
  // four columns' loads in flight a thread
  const int step = static_cast<int>(blockDim.x);
  for (int c0 = static_cast<int>(threadIdx.x); c0 < n_out; c0 += 4 * step) {
    float gate[4], up[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + i * step;
      if (c < n_out) {
        gate[i] = ld_global(r + c);
        up[i] = ld_global(r + n_out + c);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + i * step;
      if (c >= n_out) break;
      const float y = silu_mul(gate[i], up[i]);
      if constexpr (std::is_same<T, float>::value)
        h[row * ldd + c] = y;
      else if constexpr (std::is_same<T, __half>::value)
        h[row * ldd + c] = __float2half_rn(y);
      else
        h[row * ldd + c] = __float2bfloat16_rn(y);
    }
  }
}

template <int NC>
int pair_smem(int G) {
  constexpr int S = stages_of(NC);
  return 1024 + S * static_cast<int>(Layout<NC>::kStage) + 8 * (2 * S + 4) + 16 + 4 * (3 * G + 2);
}

using PairKernel = void (*)(Fp4GemmParams);

PairKernel pick_pair(int nc, int format, bool sw) {
  if (sw) return format == kNvfp4 ? fp4_pair_kernel<2, kNvfp4, true> : fp4_pair_kernel<2, kMxfp4, true>;
  if (nc == 2) return format == kNvfp4 ? fp4_pair_kernel<2, kNvfp4, false> : fp4_pair_kernel<2, kMxfp4, false>;
  return format == kNvfp4 ? fp4_pair_kernel<1, kNvfp4, false> : fp4_pair_kernel<1, kMxfp4, false>;
}

// Co-resident pairs of a kernel at the largest shared memory, and its
// attribute set, once per device.
bwg_status pair_clusters(PairKernel k, int nc, const Runtime& rt, int* clusters) {
  struct Key {
    PairKernel k;
    int dev;
  };
  static std::mutex mu;
  static struct {
    Key key;
    int clusters;
  } seen[64 * 6];
  static int n_seen = 0;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < n_seen; ++i)
    if (seen[i].key.k == k && seen[i].key.dev == rt.device) {
      *clusters = seen[i].clusters;
      return BWG_OK;
    }
  const void* fn = reinterpret_cast<const void*>(k);
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, rt.max_smem) != cudaSuccess) {
    cudaGetLastError();
    return BWG_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kPairThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(rt.max_smem);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, fn) != cudaSuccess) {
    cudaGetLastError();
    return BWG_ERR_CUDA;
  }
  // the register split only completes if the CTA was launched with at least the
  // registers that it hands out
  if (nc == 2 && static_cast<uint32_t>(fa.numRegs) * kPairThreads < kRegsControl * 128u + kRegsEpilogue * 256u)
    return BWG_ERR_UNSUPPORTED;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = rt.sm_count / 2;
  }
  if (n_seen < static_cast<int>(sizeof(seen) / sizeof(seen[0]))) {
    seen[n_seen].key = Key{k, rt.device};
    seen[n_seen].clusters = n;
    ++n_seen;
  }
  *clusters = n;
  return BWG_OK;
}

// Kernel of a dense product: 0 the few-rows kernel, 1 or 2 pairs with as many
// weight blocks a CTA.  Up to 128 rows the first; above, the one whose rounds of
// tiles take the least time: a start, and for each round its k-blocks and a
// tile's switch, or the epilogue where that is longer (in 10 ns, fitted to 132
// sizes of 200 to 4096 rows, where the fastest is taken but for 0.2% on average;
// all of them NVFP4 with BF16 output: MXFP4's k-blocks in pairs are a tenth
// shorter and FP32 output stores twice the bytes).
// The few-rows kernel is ready sooner and splits tiles: 200 rows of 4096 x 7168
// 9.1 us against 11.6 and 18.2; 960 rows of 4096 x 2048 8.2, 9.6 and 10.5.  One
// block has the shorter k-blocks (1900 rows of 4096 x 7168 32.4, 26.5 and 32.3),
// two cost the least per product (4096 rows of 8192 x 8192 125, 88 and 85).
int dense_kernel(int M, int N, int kb, int sm_count) {
  if (M <= kSmallMaxRows) return 0;
  auto rounds = [&](long long rows, long long cols, int workers) {
    const long long tiles = (M + rows - 1) / rows * ((N + cols - 1) / cols);
    return (tiles + workers - 1) / workers;
  };
  const long long few = 320 + rounds(128, 128, sm_count) * std::max(24 * kb + 45, 150);
  const long long one = 470 + rounds(kTok, 256, sm_count / 2) * std::max(25 * kb + 55, 175);
  const long long two = 520 + rounds(kTok, 512, sm_count / 2) * std::max(44 * kb + 180, 310);
  return few <= one && few <= two ? 0 : one <= two ? 1 : 2;
}

// Weight blocks a CTA for a plain grouped product.  A tile of two blocks takes
// 1.9 times as long as one of one block, but a pair's last round of tiles is
// then twice as coarse (4096 x 4096 NVFP4: 4096 tokens x 8 of 32 experts 183 us
// with two, 194 with one; 16 tokens 49.4 and 47.4, one token 14.6 and 17.6).
int grouped_blocks(int M, int N, int groups, int pairs) {
  // a ragged group ends on half a tile on average
  const long long rows = (M + kTok - 1LL) / kTok + groups / 2;
  const long long one = (rows * ((N + 255) / 256) + pairs - 1) / pairs;
  const long long two = (rows * ((N + 511) / 512) + pairs - 1) / pairs;
  return 19 * two <= 10 * one ? 2 : 1;
}

// Kernel of a product: 0 the few-rows kernel, else pairs of 1 or 2 weight blocks a
// CTA.  groups: 0 for the dense product.  n_out: columns of the result.
int product_kernel(int M, int n_out, int K, int groups, bool swiglu, int sm_count) {
  if (swiglu) return 2;
  if (groups > 0) return grouped_blocks(M, n_out, groups, sm_count / 2);
  return dense_kernel(M, n_out, (K + kKCols - 1) / kKCols, sm_count);
}

struct Fp4Operand {
  const void* codes;
  const void* scales;
  const float* global;
  int n_global;
};

bool fp4_maps(Fp4GemmParams* p, const Fp4Operand& a, const Fp4Operand& b, int M, int N_w, int K, int format, int G,
              int a_row_blocks) {
  const uint64_t row = static_cast<uint64_t>(K / 2);
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, u32 = CU_TENSOR_MAP_DATA_TYPE_UINT32;
  const uint64_t kt = static_cast<uint64_t>(fp4_k_tiles(K, format));
  const uint32_t kbox = format == kNvfp4 ? 4 : 2;
  const uint64_t wd[3] = {row, static_cast<uint64_t>(N_w), static_cast<uint64_t>(G)};
  const uint64_t ws[2] = {row, row * static_cast<uint64_t>(N_w)};
  const uint32_t wb[3] = {kKBytes, 128, 1};
  const uint64_t ad[2] = {row, static_cast<uint64_t>(M)};
  const uint32_t ab[2] = {kKBytes, kTok / 2};
  const uint64_t sd[3] = {128, kt, static_cast<uint64_t>(G) * static_cast<uint64_t>(p->w_blocks)};
  const uint64_t ss[2] = {kScaleTileBytes, kt * kScaleTileBytes};
  const uint32_t sb[3] = {128, kbox, 1};
  const uint64_t asd[3] = {128, kt, static_cast<uint64_t>(a_row_blocks)};
  const uint32_t asb[3] = {128, kbox, 2};
  return runtime_map(&p->map_w, b.codes, u8, 3, wd, ws, wb, CU_TENSOR_MAP_SWIZZLE_128B) &&
         runtime_map(&p->map_a, a.codes, u8, 2, ad, &row, ab, CU_TENSOR_MAP_SWIZZLE_128B) &&
         runtime_map(&p->map_ws, b.scales, u32, 3, sd, ss, sb, CU_TENSOR_MAP_SWIZZLE_NONE) &&
         runtime_map(&p->map_as, a.scales, u32, 3, asd, ss, asb, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Cluster size of a few-rows call, with all clusters co-resident; 1 where the
// tiles alone fill half of the SMs.  A k-block is about 0.21 us, the sum of a
// split tile's partials 0.7 us and 1.25 for each 100 rows.
int small_split(int tiles, int rows, int kb, int sm_count, const int* clusters) {
  if (2 * tiles > sm_count) return 1;
  int best = 1, least = 21 * kb;
  for (int f = 2; f <= kSmallMaxSplit; ++f) {
    const int cost = 21 * ((kb + f - 1) / f) + 70 + rows * 5 / 4;
    if (tiles <= clusters[f] && f <= kb && cost < least) {
      best = f;
      least = cost;
    }
  }
  return best;
}

bwg_status run_small(const Fp4Operand& a, const Fp4Operand& b, void* D, int M, int N, int K, int ldd, int format,
                     int out_dtype, const Runtime& rt, cudaStream_t stream) {
  using Kernel = void (*)(Fp4SmallParams);
  const bool many = M > kSmallMaxRows;
  const Kernel k = format == kNvfp4 ? (many ? fp4_small_kernel<kNvfp4, true> : fp4_small_kernel<kNvfp4, false>)
                                    : (many ? fp4_small_kernel<kMxfp4, true> : fp4_small_kernel<kMxfp4, false>);
  // co-resident clusters by size, once per device (every call of this kernel
  // takes more than half of an SM's shared memory)
  static std::mutex mu;
  static struct {
    bool ready;
    int clusters[kSmallMaxSplit + 1];
  } seen[64][2][2];
  if (rt.device >= 64) return BWG_ERR_UNSUPPORTED;
  auto& info = seen[rt.device][format][many];
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!info.ready) {
      const void* fn = reinterpret_cast<const void*>(k);
      if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, rt.max_smem) != cudaSuccess) {
        cudaGetLastError();
        return BWG_ERR_CUDA;
      }
      cudaLaunchConfig_t cfg = {};
      cfg.blockDim = dim3(kSmallThreads, 1, 1);
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      for (int f = 2; f <= kSmallMaxSplit; ++f) {
        cfg.gridDim = dim3(static_cast<unsigned>(f), 1, 1);
        cfg.dynamicSmemBytes = static_cast<size_t>(rt.max_smem);
        attr[0].val.clusterDim.x = static_cast<unsigned>(f);
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
          cudaGetLastError();
          n = 0;
        }
        info.clusters[f] = n;
      }
      info.ready = true;
    }
  }
  Fp4SmallParams p;
  std::memset(&p, 0, sizeof(p));
  p.n = std::min(kSmallMaxRows, (M + 15) & ~15);
  p.row_tiles = (M + kSmallMaxRows - 1) / kSmallMaxRows;
  const uint64_t row = static_cast<uint64_t>(K / 2);
  const uint64_t kt = static_cast<uint64_t>(fp4_k_tiles(K, format));
  const uint32_t kbox = format == kNvfp4 ? 4 : 2;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, u32 = CU_TENSOR_MAP_DATA_TYPE_UINT32;
  const uint64_t wd[3] = {row, static_cast<uint64_t>(N), 1}, ws[2] = {row, row * static_cast<uint64_t>(N)};
  const uint32_t wb[3] = {kKBytes, 128, 1};
  const uint64_t ad[2] = {row, static_cast<uint64_t>(M)};
  const uint32_t ab[2] = {kKBytes, static_cast<uint32_t>(p.n)};
  const uint64_t ss[2] = {kScaleTileBytes, kt * kScaleTileBytes};
  const uint64_t wsd[3] = {128, kt, static_cast<uint64_t>(pad128(N) / 128)}, asd[3] = {128, kt, static_cast<uint64_t>(p.row_tiles)};
  const uint32_t sb[3] = {128, kbox, 1};
  if (!runtime_map(&p.map_w, b.codes, u8, 3, wd, ws, wb, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !runtime_map(&p.map_a, a.codes, u8, 2, ad, &row, ab, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !runtime_map(&p.map_ws, b.scales, u32, 3, wsd, ss, sb, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !runtime_map(&p.map_as, a.scales, u32, 3, asd, ss, sb, CU_TENSOR_MAP_SWIZZLE_NONE))
    return BWG_ERR_CUDA;
  p.err = rt.err;
  p.timeout_ns = rt.timeout_ns;
  p.tx_extra = rt.tx_extra;
  p.a_global = a.global;
  p.b_global = b.global;
  p.d = D;
  p.ldd = ldd;
  p.M = M;
  p.N = N;
  p.num_k_blocks = (K + kKCols - 1) / kKCols;
  p.last_steps = (K - (p.num_k_blocks - 1) * kKCols + 63) / 64;
  p.tiles = (N + 127) / 128 * p.row_tiles;
  p.split = small_split(p.tiles, std::min(M, kSmallMaxRows), p.num_k_blocks, rt.sm_count, info.clusters);
  p.out_dtype = out_dtype;
  const int stage = static_cast<int>(small_stage_bytes(p.n));
  const int tail = 1024 + 8 * (2 * kSmallMaxStages + 4) + 16;
  p.stages = std::min(kSmallMaxStages, (rt.max_smem - tail) / stage);
  if (p.stages < 2) return BWG_ERR_UNSUPPORTED;
  const int grid = p.split > 1 ? p.tiles * p.split : std::min(p.tiles, rt.sm_count);
  return runtime_status(launch_overlapped(k, static_cast<unsigned>(grid), static_cast<unsigned>(small_threads(p.n)),
                                          static_cast<size_t>(p.stages * stage + tail), stream,
                                          static_cast<unsigned>(p.split), p));
}

bool aligned16(const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; }

bwg_status run_fp4_gemm(const Fp4Operand& a, const Fp4Operand& b, void* D, int M, int N, int K, int ldd, int format,
                        const int* offsets, int G, int out_dtype, bool swiglu, cudaStream_t stream) {
  if (out_dtype != BWG_OUT_BF16 && out_dtype != BWG_OUT_FP32 && out_dtype != BWG_OUT_FP16) return BWG_ERR_INVALID_ARG;
  if (format != kNvfp4 && format != kMxfp4) return BWG_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || K < 0 || G < 0) return BWG_ERR_INVALID_ARG;
  if (K % 32 != 0) return BWG_ERR_ALIGNMENT;
  if (M == 0 || N == 0 || G == 0) return BWG_OK;
  const int n_out = swiglu ? N / 2 : N;
  if (D == nullptr || ldd < n_out) return BWG_ERR_INVALID_ARG;
  if (format == kMxfp4 && (a.global != nullptr || b.global != nullptr)) return BWG_ERR_INVALID_ARG;
  if (b.global != nullptr && b.n_global != 1 && b.n_global != G) return BWG_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(D) & (out_dtype == BWG_OUT_FP32 ? 3u : 1u)) return BWG_ERR_ALIGNMENT;
  if (K > 0) {
    if (a.codes == nullptr || a.scales == nullptr || b.codes == nullptr || b.scales == nullptr)
      return BWG_ERR_INVALID_ARG;
    if (!aligned16(a.codes) || !aligned16(a.scales) || !aligned16(b.codes) || !aligned16(b.scales))
      return BWG_ERR_ALIGNMENT;
  }
  if (G > kFp4MaxGroups || M > kFp4MaxSize || N > kFp4MaxSize || K > kFp4MaxSize) return BWG_ERR_UNSUPPORTED;
  Runtime rt;
  bwg_status st = runtime_device(&rt);
  if (st != BWG_OK) return st;
  if (K == 0) {
    const int elt = out_dtype == BWG_OUT_FP32 ? 4 : 2;
    if (offsets == nullptr) return runtime_status(launch_zero_fill(D, M, n_out, ldd, elt, stream));
    return runtime_status(launch_overlapped(fp4_zero_rows_kernel, static_cast<unsigned>(M), 128, 0, stream, 1, offsets, G,
                                            M, static_cast<uint8_t*>(D), static_cast<size_t>(ldd) * elt,
                                            static_cast<size_t>(n_out) * elt, rt.err));
  }
  const int nc = product_kernel(M, n_out, K, offsets != nullptr ? G : 0, swiglu, rt.sm_count);
  if (nc == 0)
    return run_small(a, b, D, M, N, K, ldd, format, out_dtype, rt, stream);
  Fp4GemmParams p;
  std::memset(&p, 0, sizeof(p));
  const long long tok_tiles = (M + kTok - 1LL) / kTok + (offsets != nullptr ? G : 0);  // at most
  p.w_blocks = pad128(N) / 128;
  const int a_rows = offsets != nullptr ? static_cast<int>((M + 127LL * std::min(G, M)) / 128) : pad128(M) / 128;
  if (!fp4_maps(&p, a, b, M, N, K, format, G, a_rows)) return BWG_ERR_CUDA;
  p.err = rt.err;
  p.timeout_ns = rt.timeout_ns;
  p.tx_extra = rt.tx_extra;
  p.offsets = offsets;
  p.a_global = a.global;
  p.b_global = b.global;
  p.b_globals = b.n_global;
  p.d = D;
  p.ldd = ldd;
  p.M = M;
  p.N = n_out;
  p.G = G;
  p.num_k_blocks = (K + kKCols - 1) / kKCols;
  p.last_steps = (K - (p.num_k_blocks - 1) * kKCols + 63) / 64;
  const int w_rows = swiglu ? 256 : 256 * nc;
  p.num_w_tiles = (n_out + w_rows - 1) / w_rows;
  p.swiglu_up = n_out;
  p.out_dtype = out_dtype;
  p.group_m = 8;
  const int smem = nc == 2 ? pair_smem<2>(G) : pair_smem<1>(G);
  if (smem > rt.max_smem) return BWG_ERR_UNSUPPORTED;
  const PairKernel k = pick_pair(nc, format, swiglu);
  int clusters = 0;
  if ((st = pair_clusters(k, nc, rt, &clusters)) != BWG_OK) return st;
  // every group adds at most one partial tile of rows
  const long long most = tok_tiles * p.num_w_tiles;
  const int grid = 2 * static_cast<int>(std::min<long long>(most, clusters));
  return runtime_status(launch_overlapped(k, static_cast<unsigned>(grid), kPairThreads,
                                          static_cast<size_t>(smem), stream, 2, p));
}

// Grouped product with SwiGLU where the up half starts inside a tile of
// scales: the FP32 product into the workspace, then the activation.
bwg_status run_swiglu_two_steps(const Fp4Operand& a, const Fp4Operand& b, void* H, int M, int N, int K, int ldh,
                                int format, const int* offsets, int G, int out_dtype, void* workspace,
                                cudaStream_t stream) {
  if (out_dtype != BWG_OUT_BF16 && out_dtype != BWG_OUT_FP32 && out_dtype != BWG_OUT_FP16) return BWG_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || N % 2 != 0 || K < 0 || G < 0) return BWG_ERR_INVALID_ARG;
  if (M == 0 || N == 0 || G == 0) return BWG_OK;
  if (H == nullptr || workspace == nullptr || ldh < N / 2) return BWG_ERR_INVALID_ARG;
  if (!aligned16(workspace) || (reinterpret_cast<uintptr_t>(H) & (out_dtype == BWG_OUT_FP32 ? 3u : 1u)))
    return BWG_ERR_ALIGNMENT;
  const bwg_status st =
      run_fp4_gemm(a, b, workspace, M, N, K, N, format, offsets, G, BWG_OUT_FP32, false, stream);
  if (st != BWG_OK) return st;
  const float* x = static_cast<const float*>(workspace);
  const int n = N / 2, threads = std::min(256, (n + 31) / 32 * 32);
  const unsigned blocks = static_cast<unsigned>(M);
  cudaError_t e;
  if (out_dtype == BWG_OUT_FP32)
    e = launch_overlapped(fp4_swiglu_kernel<float>, blocks, static_cast<unsigned>(threads), 0, stream, 1, x, offsets, G, n,
                          static_cast<long long>(ldh), static_cast<float*>(H));
  else if (out_dtype == BWG_OUT_FP16)
    e = launch_overlapped(fp4_swiglu_kernel<__half>, blocks, static_cast<unsigned>(threads), 0, stream, 1, x, offsets, G, n,
                          static_cast<long long>(ldh), static_cast<__half*>(H));
  else
    e = launch_overlapped(fp4_swiglu_kernel<__nv_bfloat16>, blocks, static_cast<unsigned>(threads), 0, stream, 1, x, offsets, G, n,
                          static_cast<long long>(ldh), static_cast<__nv_bfloat16*>(H));
  return runtime_status(e);
}

}  // namespace
}  // namespace bwg

using namespace bwg;

extern "C" {

int bwg_fp4_kernel(int M, int N, int K, int G, int swiglu, int sm_count) {
  if (M < 1 || N < 1 || K < 1 || G < 0 || sm_count < 2 || M > kFp4MaxSize || N > kFp4MaxSize || K > kFp4MaxSize) return -1;
  return product_kernel(M, swiglu && N % 256 == 0 ? N / 2 : N, K, G, swiglu && N % 256 == 0, sm_count);
}

bwg_status gemm_fp4(const void* A, const void* A_scales, const float* A_global, const void* B, const void* B_scales,
                    const float* B_global, int format, void* D, int M, int N, int K, int ldd, int out_dtype,
                    void* stream) {
  return run_fp4_gemm(Fp4Operand{A, A_scales, A_global, 1}, Fp4Operand{B, B_scales, B_global, 1}, D, M, N, K, ldd,
                      format, nullptr, 1, out_dtype, false, static_cast<cudaStream_t>(stream));
}

bwg_status grouped_gemm_fp4(const void* A, const void* A_scales, const float* A_global, const void* B,
                            const void* B_scales, const float* B_global, int n_global, int format, void* D,
                            const int* group_offsets, int G, int M_total, int N, int K, int ldd, int out_dtype,
                            int swiglu, void* workspace, void* stream) {
  if (M_total > 0 && N > 0 && G > 0 && group_offsets == nullptr) return BWG_ERR_INVALID_ARG;
  const Fp4Operand a{A, A_scales, A_global, 1}, b{B, B_scales, B_global, n_global};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (swiglu && N % 256 != 0)
    return run_swiglu_two_steps(a, b, D, M_total, N, K, ldd, format, group_offsets, G, out_dtype, workspace, s);
  return run_fp4_gemm(a, b, D, M_total, N, K, ldd, format, group_offsets, G, out_dtype, swiglu != 0, s);
}

}  // extern "C"
