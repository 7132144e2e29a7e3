// Grouped products on the tensor cores (tcgen05, 16-bit inputs, 32-bit sums in tensor memory).
//
// One kernel computes D[m, j] = sum_k A[m, k] B[j, k] for five products.  The dense, always long
// side is M (weight rows or columns); the ragged side, the rows of a group, is N, because the
// instruction takes any N that is a multiple of 16: a group of 5 rows costs an instruction of 16
// columns, not a tile of 128, and the last tile of each group only what it holds.
//
//   mode      A (M side)                      B (N side)                       contracted k
//   Forward   w[g] rows                       x rows, gathered or in order     columns of x
//   Gated     64 gate rows + 64 up rows       x rows, gathered                 columns of x
//   Dx        w[g]^T (columns of w[g])        dy rows                          rows of w[g]
//   Dw        x^T (columns of x, in order)    dy^T (columns of dy)             the group's positions
//   Adapted   w rows, then b[i] rows          x rows, then v rows of adapter i columns of x, then rank
//
// Operands go to shared memory in 64-deep slices by bulk copies: 128-byte swizzled boxes.  Rows in any
// order come by gathering copies, four rows each, about 40 cycles from one warp where the matrix instruction
// takes 8 for them.  They serve tiles of at most 128 rows where groups have few rows (mma_gathers()) and the ends of
// groups; for more rows x is laid out in group order first.
// A gathered row index past the matrix reads as zeros: that masks the positions behind a group's
// end (Dw, where they are contracted, on both operands, so that a NaN there cannot leak) and, in Adapted,
// the tokens of other adapters.
//
// Thirteen warps: four producers (a warp issues its lanes' copies one after the other, so a slice's copies
// are dealt over four), an issuer (matrix instructions, one thread), two sets of four that empty the
// accumulators while the next tile is computed into the other half of tensor memory (the last tile's
// emptying is not hidden: two sets halve it).  The accumulator's lanes are consecutive columns of the
// output, so a warp's store is contiguous.  Persistent blocks.
//
// Pairs: tiles of 256 rows are shared by two blocks (cta_group::2): each holds half of A and half of B, so
// an SM fetches 32 KB per slice of 512 cycles instead of 48.  A stage holds two slices: with one, the issuer's
// barrier round per slice (about 450 cycles) took as long as the slice's instructions (368 -> 315 us below).
//
// Split: where there are fewer tiles than half the SMs, the blocks of a cluster share a tile's contracted
// range, send each other their part of the sums through distributed shared memory and add them up
// in the order of their ranks.
//
// Measured on GB300 (of the measured 1935 TFLOP/s and 6.69 TB/s): 65536 rows, 32 unequal groups, 2048 x 2048:
// forward 315 us with 32-bit rows (1745 TFLOP/s, 90%; equal groups 303 us, the library's dense batched product 280 us),
// 348 us with 16-bit rows and their marks (k_group_settle.cu adds 1.58 ms in bf16), dx 344 us
// (83%, 32-bit rows out), dw 336 us (85%); tensor pipe 73% busy, the rest is barrier rounds and the epilogue's
// stores (20 us of 303).  Gated, 49152 rows, 64 groups, 2048 x 2048: 267 us (1540 TFLOP/s, 80%).  Adapted, 8192
// rows, 4096 x 4096, rank 64: 165 us (1760 TFLOP/s, 91%).  A layer of eight tokens and 64 experts reads its
// weights at 90% of the copy rate: 67 us; what is missing is the last wave of tiles and the first one's set-up.
//
// Every wait is bounded: a role that gives up sets the status word, the others see it, copies in
// flight are drained, tensor memory is freed, the kernel returns.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "group_mma.h"
#include "tc.cuh"

namespace sg {

namespace {

constexpr int kProducers = 4;      // producer warps; warp 4 issues, warps 5 to 12 are the epilogue
constexpr int kSets = 2;           // sets of four epilogue warps: every other 32 columns each
constexpr int kEpilogue = 128 * kSets;
constexpr int kThreads = 32 * (kProducers + 1) + kEpilogue;
constexpr int kDeep = 64;          // contracted elements of a slice: 128 bytes, one swizzle row
constexpr int kMaxStages = 12;
constexpr int kABytes = 128 * 128; // A's part of a stage: 128 rows of 128 bytes
constexpr int kBox = 64 * 128;     // a 64 x 64 box
constexpr int kTmemCols = 512;
constexpr int kSplitTile = 64;     // widest tile that is split: its sums (128 x 64, 32 KB) meet in the stages of half an SM
constexpr int kSmemMost = 227 * 1024;

struct Control {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  int failed[2];                   // a role gave up; polls allowed to a wait
  int go[kSets][2];                // Gated: whether the four warps of a set take the next tile
  int last[kMaxStages];            // 1: the stage holds the last slice of its tile
  int scan[33];
  int first[kMaxGroups + 1];       // first position of each group (clamped to [0, slots])
  int tiles[kMaxGroups + 1];       // N-side tiles of the groups before each
};

// Gated: columns that the gate and up warps of a set exchange, by turns
struct Swap {
  float v[kSets][2][4][8][32];
};

// whether two 32-bit values round to different numbers of the type
template <typename T>
__device__ __forceinline__ bool rounds_apart(float a, float b);
template <>
__device__ __forceinline__ bool rounds_apart<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return __bfloat16_as_ushort(v.x) != __bfloat16_as_ushort(v.y);
}
template <>
__device__ __forceinline__ bool rounds_apart<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return __half_as_ushort(__low2half(v)) != __half_as_ushort(__high2half(v));
}

struct Tile {
  int g;       // group
  int m0;      // first M index
  int j0;      // first position (Dw: first column of dy)
  int n;       // N indices that count
  int k0, k;   // contracted range: first position and length (Dw), else 0 and the depth
};

}  // namespace

// Adapted: the products of a tile's adapters go to all of its columns, the tokens of others meeting them with zeros.
// Zero times an infinite or NaN b is NaN, so a sum that is not finite is formed again, in 32 bits, from what belongs to
// its token, where the tile holds an adapter that is not the token's own.  A warp does it: `lanes` are those whose sum
// at `token` is not finite, m0 the column of lane 0; lane i gets its sum in *sum if its bit is in the answer.
// 8192 rows, 4096 x 4096, rank 64, 16 adapters (198 us): 1.3 ms with one infinite value in an adapter, 9.9 ms with an
// adapter of NaN.
template <typename T>
__device__ __noinline__ uint32_t own_sums(const MmaArgs& p, int j0, int n, int token, int m0, uint32_t lanes, float* sum) {
  const int lane = threadIdx.x & 31;
  auto id_of = [&](int t) {
    const int id = p.ids[t];
    return id >= 0 && id < p.adapters ? id : -1;
  };
  const int own = id_of(token);
  bool others = false;
  for (int j = lane; j < n; j += 32) {
    const int id = id_of(j0 + j);
    others = others || (id >= 0 && id != own);
  }
  if (!__any_sync(0xffffffffu, others)) return 0u;
  pdl_wait();  // v is the kernel's before this one
  // the 8-deep pieces first, first + step, ... of a scalar product; rows start on 16 bytes
  auto dot = [&](float acc, const void* a, int64_t a_at, const void* b, int64_t b_at, int depth, int first, int step) {
    const T *u = static_cast<const T*>(a) + a_at, *v = static_cast<const T*>(b) + b_at;
#pragma unroll 4
    for (int k = 8 * first; k + 8 <= depth; k += 8 * step) {
      const uint4 x = *reinterpret_cast<const uint4*>(u + k), y = *reinterpret_cast<const uint4*>(v + k);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        acc = fmaf(to_f32(reinterpret_cast<const T*>(&x)[e]), to_f32(reinterpret_cast<const T*>(&y)[e]), acc);
    }
    if (depth / 8 % step == first)
      for (int k = depth / 8 * 8; k < depth; ++k) acc = fmaf(to_f32(u[k]), to_f32(v[k]), acc);
    return acc;
  };
  auto whole = [&](int l, int first, int step) {
    float acc = dot(0.0f, p.x, token * p.x_stride, p.w, (m0 + l) * p.w_stride, p.depth, first, step);
    if (own >= 0) acc = dot(acc, p.v, token * p.v_stride, p.b, own * p.b_group + (m0 + l) * p.b_stride, p.rank, first, step);
    return acc;
  };
  if (__popc(lanes) > 8) {  // each lane its own sum
    if ((lanes >> lane) & 1u) *sum = whole(lane, 0, 1);
    __syncwarp();
  } else {  // all lanes one sum after the other
    for (uint32_t left = lanes; left; left &= left - 1) {
      const int l = __ffs(left) - 1;
      const float acc = warp_sum(whole(l, lane, 32));
      if (lane == l) *sum = acc;
    }
  }
  return lanes;
}

__device__ __forceinline__ bool not_finite(uint32_t bits) { return (bits & 0x7fffffffu) >= 0x7f800000u; }

struct MmaMaps {
  CUtensorMap a, b, c, d;  // Forward, Dx: weights, rows (gathered: also in boxes); Dw: x, dy, then rows of dy and of x; Adapted: w, x, b[i], v rows
};

template <int MODE, bool PAIR, bool SPLIT>
__global__ void __launch_bounds__(kThreads, SPLIT ? 2 : 1) k_group_mma(const __grid_constant__ MmaMaps maps,
                                                           const __grid_constant__ MmaArgs p) {
  using namespace tc;
  extern __shared__ char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  Control& c = *reinterpret_cast<Control*>(smem_raw + (base - smem_u32(smem_raw)) + p.stages * p.stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0u;          // block of the pair
  const int part = SPLIT ? static_cast<int>(cluster_rank()) : 0, parts = SPLIT ? p.split : 1;  // of the contracted range
  const uint32_t tmem_cols = SPLIT ? kSplitTile : kTmemCols;
  constexpr int kSide = PAIR ? 2 : 1;
  constexpr int kSub = SPLIT ? 1 : 2;  // slices of a stage
  constexpr bool kDw = MODE == kMmaDw;
  volatile int* failed = c.failed;

  // ---- set-up: barriers, tensor memory, the groups' first positions and tile counts -----------
  if (warp == 0) {
    if (lane < p.stages) {
      // tests: an arrival that never comes, on the first stage of block 0
      mbar_init(smem_u32(&c.full[lane]), p.hold && blockIdx.x == 0 && lane == 0 ? 2 : 1);
      mbar_init(smem_u32(&c.empty[lane]), 1);
    } else if (lane < p.stages + 2) {
      mbar_init(smem_u32(&c.acc_full[lane - p.stages]), 1);
      mbar_init(smem_u32(&c.acc_empty[lane - p.stages]), kEpilogue * kSide);
    } else if (lane == 31) {
      mbar_init(smem_u32(&c.drain), 1);
      c.failed[0] = 0;
      c.failed[1] = static_cast<int>(p.polls);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (warp == 1 && lane == 0) {
    prefetch_map(&maps.a);
    prefetch_map(&maps.b);
    prefetch_map(&maps.c);
    prefetch_map(&maps.d);
  }
  if (PAIR) cluster_sync();  // both blocks run before one allocates in both
  if (warp == kProducers) tmem_alloc<PAIR>(smem_u32(&c.tmem), tmem_cols);
  // `early`: the kernel before this one (of the same call, itself started after everything before it was
  // complete) makes only the rows of B, or v.  Weights, offsets and ids are read while it ends.
  if (!p.early) {
    pdl_wait();
    pdl_go();
  }
  // offsets are used as a non-decreasing sequence inside [0, slots], whatever the array holds
  {
    int run = 0;
    for (int g0 = 0; g0 < p.groups; g0 += kThreads) {
      const int g = g0 + static_cast<int>(threadIdx.x);
      int lo = 0, hi = 0;
      if (g < p.groups) {
        lo = p.offsets ? min(max(p.offsets[g], 0), p.slots) : 0;
        hi = p.offsets ? min(max(p.offsets[g + 1], lo), p.slots) : p.slots;
        c.first[g] = lo;
        if (g == p.groups - 1) c.first[p.groups] = hi;
      }
      if (kDw) continue;
      const int n = (hi - lo + p.tile_n - 1) / p.tile_n;
      int top = 0;
      const int before = run + block_incl_scan(n, c.scan, &top) - n;
      if (g < p.groups) c.tiles[g] = before;
      run += top;
    }
    if (threadIdx.x == 0) c.tiles[p.groups] = run;
  }
  fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();
  fence_after();
  const uint32_t tmem = c.tmem;
  const int m_per_tile = (MODE == kMmaGated ? 64 : 128) * kSide;
  const int mt = (p.m + m_per_tile - 1) / m_per_tile;
  const int nt = kDw ? (p.n + p.tile_n - 1) / p.tile_n : 0;
  const int worker = static_cast<int>(PAIR ? blockIdx.x >> 1 : SPLIT ? blockIdx.x / parts : blockIdx.x);
  const int workers = static_cast<int>(PAIR ? gridDim.x >> 1 : SPLIT ? gridDim.x / parts : gridDim.x);

  // Tiles in the order m fastest, then the N side, group by group: blocks that run at the same time share a
  // group's weights and rows in L2.  (All full tiles first, then the groups' part tiles, balances the blocks
  // better but reads the weights twice.)  A walk keeps its place; no division per tile.
  const int all_tiles = kDw ? p.groups * nt : c.tiles[p.groups];
  struct Walk {
    int m, r, g;
  };
  const int step_m = workers % mt, step_r = workers / mt;
  auto start = [&]() { return Walk{worker % mt, worker / mt, 0}; };
  auto advance = [&](Walk& w) {
    w.m += step_m;
    w.r += step_r;
    if (w.m >= mt) {
      w.m -= mt;
      ++w.r;
    }
  };
  auto tile_of = [&](Walk& w) {
    Tile t;
    t.m0 = w.m * m_per_tile;
    if (kDw) {
      t.g = w.r / nt;
      t.j0 = (w.r - t.g * nt) * p.tile_n;
      t.n = min(p.n - t.j0, p.tile_n);
      t.k0 = c.first[t.g];
      t.k = max(c.first[t.g + 1] - t.k0, 0);
    } else {
      while (w.g + 1 < p.groups && c.tiles[w.g + 1] <= w.r) ++w.g;
      const int lo = c.first[w.g], hi = p.offsets ? min(max(p.offsets[w.g + 1], lo), p.slots) : p.slots;
      t.g = w.g;
      t.j0 = lo + (w.r - c.tiles[w.g]) * p.tile_n;
      t.n = min(hi - t.j0, p.tile_n);
      t.k0 = 0;
      t.k = p.depth;
    }
    return t;
  };
  // columns of the instruction: a multiple of 16 per block of the pair
  auto columns = [&](int n) { return (n + 16 * kSide - 1) / (16 * kSide) * (16 * kSide); };

  if (warp < kProducers) {
    // ---- producers ---------------------------------------------------------------------------------
    int s = 0;
    uint32_t phase = 0;
    bool ok = true, waited = !p.early;
    auto wait_before = [&]() {
      if (waited) return;
      pdl_wait();
      pdl_go();
      waited = true;
    };
    for (Walk w = start(); w.r < all_tiles && ok; advance(w)) {
      const Tile t = tile_of(w);
      const int cols = columns(t.n), half = cols / kSide;
      const int jr = t.j0 + static_cast<int>(rank) * half;  // first N index of this block
      // four rows that this lane gathers: a quad of this block's N side
      const int quad = lane * kProducers + warp;
      const bool gather = (MODE == kMmaForward || MODE == kMmaGated) && p.gather;
      int4 mine = make_int4(0, 0, 0, 0);
      if (gather && quad * 4 < half) {
        int r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = jr + quad * 4 + e;
          const int slot = j < t.j0 + t.n ? p.order[j] : -1;
          r[e] = slot >= 0 ? min(slot / p.top_k, p.rows) : p.rows;
        }
        mine = make_int4(r[0], r[1], r[2], r[3]);
      }
      auto bar = [&]() { return PAIR ? map_rank(smem_u32(&c.full[s]), 0) : smem_u32(&c.full[s]); };
      // The first warp announces a stage's bytes, the barrier's only arrival (a copy of another warp may be done
      // before).  `units`: copies of the stage that are dealt over the warps.  A warp without one still takes
      // part, by a few bytes that it takes off itself: otherwise it could fall two rounds behind the others, and
      // a barrier's parity cannot tell two rounds from none.
      auto announce = [&](uint32_t bytes, int units) {
        const uint32_t idle = static_cast<uint32_t>(max(kProducers - units, 0)) * 16u;
        if (warp == 0 && rank == 0) mbar_expect_tx(smem_u32(&c.full[s]), (bytes + idle) * kSide);
        if (warp >= units) mbar_complete_tx(bar(), 16u);
      };
      // one stage: waits until it is free and announces its bytes; returns its address
      auto open = [&](uint32_t bytes, bool last) -> uint32_t {
        ok = mbar_wait(smem_u32(&c.empty[s]), phase ^ 1u, failed, p.err, 1u);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && lane == 0) {
          if (warp == 0) c.last[s] = last ? 1 : 0;
          announce(bytes, kProducers);
        }
        return base + s * p.stage_bytes;
      };
      auto close = [&]() {
        if (++s == p.stages) {
          s = 0;
          phase ^= 1u;
        }
      };
      const int slices = (t.k + kDeep - 1) / kDeep;
      const int q0 = SPLIT ? slices * part / parts : 0, q1 = SPLIT ? slices * (part + 1) / parts : slices;

      if (kDw) {
        const int nb = (half + 63) / 64;  // 64-column blocks of dy
        const int m0 = t.m0 + static_cast<int>(rank) * 128;
        const uint32_t bytes = static_cast<uint32_t>((2 + nb) * kBox);
        // box u: 64 columns of x (0, 1), then of dy
        auto column = [&](int u) { return u < 2 ? m0 + u * 64 : jr + (u - 2) * 64; };
        const int whole = t.k / kDeep;
        for (int q = 0; q < whole; q += kSub) {  // one lane of each warp; the others only keep count
          const int subs = min(kSub, whole - q);
          if (lane == 0 && ok) {
            ok = mbar_wait(smem_u32(&c.empty[s]), phase ^ 1u, failed, p.err, 1u);
            if (ok) {
              announce(subs * bytes, 2 + nb);
              const uint32_t fb = bar();
              for (int h = 0; h < subs; ++h)
                for (int u = warp; u < 2 + nb; u += kProducers)
                  load_2d<PAIR>(base + s * p.stage_bytes + h * p.sub_bytes + u * kBox, u < 2 ? &maps.a : &maps.b, column(u),
                                t.k0 + (q + h) * kDeep, fb);
            }
          }
          close();
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (ok && whole < slices) {  // the group ends inside the slice: rows past it read as zeros, on both sides
          const uint32_t a = open(bytes, true);
          if (!ok) break;
          const uint32_t fb = bar();
          const int u = quad >> 4;
          if (u < 2 + nb) {
            int r[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int o = whole * kDeep + (quad & 15) * 4 + e;
              r[e] = o < t.k ? t.k0 + o : p.slots;
            }
            load_rows4<PAIR>(a + u * kBox + (quad & 15) * 512, u < 2 ? &maps.d : &maps.c, column(u),
                             make_int4(r[0], r[1], r[2], r[3]), fb);
          }
          close();
        }
        continue;
      }

      // gathered rows that follow one another anyway (the tokens of one request) come in boxes
      bool boxed = !gather;
      if (MODE == kMmaForward && gather && p.runs) {
        bool follow = true;
        const int row0 = p.order[t.j0] / p.top_k;
        for (int j = lane; j < t.n; j += 32) follow = follow && p.order[t.j0 + j] / p.top_k == row0 + j;
        boxed = __all_sync(0xffffffffu, follow) != 0;
      }
      const int row_b = boxed && gather ? p.order[t.j0] / p.top_k : jr;
      const CUtensorMap* map_b = gather ? &maps.c : &maps.b;
      const int boxes = (half + p.box_rows - 1) / p.box_rows;
      // the second 64 rows of A may be none of the matrix's: the accumulator's lanes then hold nothing of use
      const int boxes_a = MODE == kMmaForward && !PAIR && t.m0 + 64 >= p.m ? 1 : 2;
      const uint32_t bytes = boxes_a * kBox + (boxed ? boxes * p.box_rows : half) * 128;
      // Adapted: the adapters of the tile's tokens (lane, lane + 32, ...), in ascending order
      int ids[8];
      auto id_of = [&](int j) {
        const int id = j < t.j0 + t.n ? p.ids[j] : -1;
        return id >= 0 && id < p.adapters ? id : -1;
      };
      auto following = [&](int before) {
        uint32_t least = 0xffffffffu;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (ids[e] > before) least = min(least, static_cast<uint32_t>(ids[e]));
        return static_cast<int>(__reduce_min_sync(0xffffffffu, least));  // -1: none left
      };
      // the next adapter of this block: all of them, or (Split) every parts-th
      auto mine_after = [&](int before, int skip) {
        int id = following(before);
        for (int e = 0; e < skip && id >= 0; ++e) id = following(id);
        return id;
      };
      int adapter = -1, quad_ids[4] = {-1, -1, -1, -1};
      if (MODE == kMmaAdapted) {
#pragma unroll
        for (int e = 0; e < 4; ++e) quad_ids[e] = quad * 4 < half ? id_of(jr + quad * 4 + e) : -1;
#pragma unroll
        for (int e = 0; e < 8; ++e) ids[e] = lane + 32 * e < t.n ? id_of(t.j0 + lane + 32 * e) : -1;
        adapter = mine_after(-1, part);
      }
      // copy u of a slice: A's two boxes, then B's; box 2 and up: none for this lane
      auto copy_a = [&](uint32_t a, int box, int k0, uint32_t fb) {
        const int m0 = t.m0 + static_cast<int>(rank) * (MODE == kMmaGated ? 64 : 128);
        if (MODE == kMmaDx) load_3d<PAIR>(a + box * kBox, &maps.a, m0 + box * 64, k0, t.g, fb);
        else if (MODE == kMmaGated) load_3d<PAIR>(a + box * kBox, &maps.a, k0, m0 + box * p.m, t.g, fb);
        else load_3d<PAIR>(a + box * kBox, &maps.a, k0, m0 + box * 64, t.g, fb);
      };
      const int box = lane == 31 ? warp : 2;
      if (!boxed) {
        wait_before();
        for (int q = q0; q < q1 && ok; q += kSub) {
          const int subs = min(kSub, q1 - q);
          const uint32_t stage = open(subs * bytes, q + subs == q1);
          if (!ok) break;
          const uint32_t fb = bar();
          for (int h = 0; h < subs; ++h) {
            const uint32_t a = stage + h * p.sub_bytes;
            if (box < boxes_a) copy_a(a, box, (q + h) * kDeep, fb);
            if (quad * 4 < half) load_rows4<PAIR>(a + kABytes + quad * 512, &maps.b, (q + h) * kDeep, mine, fb);
          }
          close();
        }
      } else {
        // fills the stage's next slice h: A's boxes, B's boxes, or both, dealt over the warps
        auto fill = [&](int q, int h, bool with_a, bool with_b, uint32_t fb) {
          const uint32_t a = base + s * p.stage_bytes + h * p.sub_bytes;
          const int k0 = (q + h) * kDeep;
          for (int u = warp; u < boxes_a + boxes; u += kProducers) {
            const int v = u - boxes_a;
            if (v < 0 && with_a) copy_a(a, u, k0, fb);
            if (v >= 0 && with_b) load_2d<PAIR>(a + kABytes + v * p.box_rows * 128, map_b, k0, row_b + v * p.box_rows, fb);
          }
        };
        int ahead = 0;  // stages whose A is on its way
        if (MODE != kMmaAdapted && !waited) {
          for (int q = q0; q < q1 && ahead < p.stages; q += kSub, ++ahead) {
            const int subs = min(kSub, q1 - q);
            if (lane == 0) {
              announce(subs * bytes, boxes_a + boxes);
              for (int h = 0; h < subs; ++h) fill(q, h, true, false, bar());
            }
            close();
          }
          s = 0;
          phase = 0;
          wait_before();
        }
        for (int q = q0; q < q1; q += kSub) {  // one lane of each warp; the others only keep count
          const int subs = min(kSub, q1 - q);
          const bool fresh = ahead-- <= 0;
          if (lane == 0 && ok) {
            if (fresh) ok = mbar_wait(smem_u32(&c.empty[s]), phase ^ 1u, failed, p.err, 1u);
            if (ok) {
              if (fresh) {
                if (MODE == kMmaAdapted && warp == 0) c.last[s] = q + subs == q1 && adapter < 0 ? 1 : 0;
                announce(subs * bytes, boxes_a + boxes);
              }
              for (int h = 0; h < subs; ++h) fill(q, h, fresh, true, bar());
            }
          }
          close();
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      // then, per adapter, its b against the v rows of its own tokens (the others' read as zeros)
      if (MODE == kMmaAdapted && adapter >= 0) wait_before();
      while (MODE == kMmaAdapted && ok && adapter >= 0) {
        const int after = mine_after(adapter, parts - 1);
        int r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = quad_ids[e] == adapter ? jr + quad * 4 + e : p.rows;
        for (int k0 = 0; k0 < p.rank && ok; k0 += kDeep) {
          const uint32_t a = open(kABytes + half * 128, k0 + kDeep >= p.rank && after < 0), b = a + kABytes;
          if (!ok) break;
          const uint32_t fb = bar();
          if (box < 2)
            load_3d<PAIR>(a + box * kBox, &maps.c, k0, t.m0 + static_cast<int>(rank) * 128 + box * 64, adapter, fb);
          if (quad * 4 < half) load_rows4<PAIR>(b + quad * 512, &maps.d, k0, make_int4(r[0], r[1], r[2], r[3]), fb);
          close();
        }
        adapter = after;
      }
    }
    // after a failure nothing consumes the stages any more: wait for the copies in flight
    if (*failed) {
      for (int q = 0; q < p.stages; ++q) {
        mbar_drain(smem_u32(&c.full[s]), phase ^ 1u, max(p.polls >> 4, 64u));
        if (++s == p.stages) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == kProducers && rank == 0) {
    // ---- issuer ----------------------------------------------------------------------------------
    int s = 0, it = 0;
    uint32_t phase = 0;
    bool ok = true;
    constexpr bool kARows = MODE == kMmaDx || MODE == kMmaDw, kBRows = MODE == kMmaDw;
    if (lane == 0) {
      for (Walk w = start(); w.r < all_tiles && ok; advance(w)) {
        const Tile t = tile_of(w);
        if (t.k == 0) continue;  // an empty group's gradient: the epilogue writes zeros
        const uint32_t idesc = instruction(p.bf16, kARows, kBRows, 128 * kSide, columns(t.n));
        const uint32_t acc = tmem + (it & 1) * p.tile_n;
        ok = mbar_wait(smem_u32(&c.acc_empty[it & 1]), ((it >> 1) & 1) ^ 1u, failed, p.err, 2u);
        fence_after();
        const int slices = (t.k + kDeep - 1) / kDeep;
        const int n = SPLIT ? slices * (part + 1) / parts - slices * part / parts : slices;
        const int paired = kDw ? t.k / kDeep : n;  // slices that come kSub to a stage
        bool last = false;
        for (int q = 0; ok && !last;) {
          ok = mbar_wait(smem_u32(&c.full[s]), phase, failed, p.err, 4u);
          if (!ok) break;
          fence_after();
          // part slices of a group and adapters' come alone
          const int subs = q < paired ? min(kSub, paired - q) : 1;
          for (int h = 0; h < subs; ++h) {
            const uint32_t a = base + s * p.stage_bytes + h * p.sub_bytes;
            mma_slice<PAIR, kARows ? 128 : 2, kBRows ? 128 : 2>(acc, operand(a, kBox), operand(a + kABytes, kBox), idesc,
                                                                q + h > 0);
          }
          q += subs;
          last = MODE == kMmaAdapted ? q >= n && c.last[s] != 0 : q == n;
          commit<PAIR>(smem_u32(&c.empty[s]));
          if (last) commit<PAIR>(smem_u32(&c.acc_full[it & 1]));
          if (++s == p.stages) {
            s = 0;
            phase ^= 1u;
          }
        }
        ++it;
      }
      if (*failed) {
        commit<PAIR>(smem_u32(&c.drain));
        mbar_drain(smem_u32(&c.drain), 0, max(p.polls >> 4, 64u));
      }
    }
    __syncwarp();
  } else if (warp > kProducers) {
    // ---- epilogue ----------------------------------------------------------------------------------
    const int quarter = warp & 3;  // the lanes of tensor memory that this warp can read
    const int ml = quarter * 32 + lane, set = (warp - kProducers - 1) >> 2;
    int it = 0, turn = 0;
    bool ok = true;
    for (Walk w = start(); w.r < all_tiles; advance(w)) {
      const Tile t = tile_of(w);
      const bool zero = t.k == 0;
      if (!zero) {
        ok = mbar_wait(smem_u32(&c.acc_full[it & 1]), (it >> 1) & 1, failed, p.err, 8u);
        ok = __all_sync(0xffffffffu, ok);
        if (MODE == kMmaGated) {  // the warps meet below: they go on together or not at all
          if ((warp - kProducers - 1) % 4 == 0 && lane == 0) c.go[set][it & 1] = ok;
          asm volatile("bar.sync %0, 128;" ::"r"(1 + set) : "memory");
          if (!c.go[set][it & 1]) break;
        } else if (!ok) {
          break;
        }
        fence_after();
      }
      if (SPLIT) break;  // the sums of the cluster's blocks meet below
      const uint32_t acc = tmem + (it & 1) * p.tile_n + (static_cast<uint32_t>(quarter * 32) << 16);
      for (int j = set * 32; j < t.n; j += 32 * kSets) {
        uint32_t r[32];
        if (zero) {
#pragma unroll
          for (int e = 0; e < 32; ++e) r[e] = 0u;
        } else {
          tmem_load32(acc + j, r);
        }
        const int n = min(32, t.n - j);
        if (MODE == kMmaGated) {
          // lanes 0..63 hold the gate's sums, 64..127 up's, of the same 64 hidden columns
          const bool up = quarter >= 2;
          Swap& swap = *reinterpret_cast<Swap*>(&c + 1);
          const int m = t.m0 + static_cast<int>(rank) * 64 + (quarter & 1) * 32 + lane;
#pragma unroll
          for (int part16 = 0; part16 < 32; part16 += 16) {  // gate warps finish columns 0..7, up warps 8..15
            float(&mine)[8][32] = swap.v[set][turn][quarter];
            const float(&theirs)[8][32] = swap.v[set][turn][quarter ^ 2];
            turn ^= 1;  // one meeting per exchange: the next one writes the other buffer
#pragma unroll
            for (int e = 0; e < 8; ++e) mine[e][lane] = __uint_as_float(up ? r[part16 + e] : r[part16 + 8 + e]);
            asm volatile("bar.sync %0, 128;" ::"r"(1 + set) : "memory");
            const int j0 = j + part16 + (up ? 8 : 0), left = t.n - j0;
            const int64_t o = static_cast<int64_t>(t.j0 + j0) * p.out_stride + m;
            auto put = [&](auto type) {
              using T = decltype(type);
              T* out = static_cast<T*>(p.out);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float other = theirs[e][lane], own = __uint_as_float(up ? r[part16 + 8 + e] : r[part16 + e]);
                // the result is rounded to 16 bits: the short exponential and division are exact enough
                const float h = gated_silu_short(up ? other : own, up ? own : other);
                if (e < left && m < p.m) out[o + e * p.out_stride] = from_f32<T>(h);
              }
            };
            if (p.out_type == SPGEMM_DTYPE_BF16) put(__nv_bfloat16());
            else put(__half());
          }
        } else {
          const int m = t.m0 + static_cast<int>(rank) * 128 + ml;
          const int64_t o = (kDw ? t.g * p.out_group : 0) + static_cast<int64_t>(t.j0 + j) * p.out_stride + m;
          if (MODE == kMmaForward && p.unsure) {
            auto mark = [&](auto type) {
              using T = decltype(type);
              uint32_t marks = 0;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float v = __uint_as_float(r[e]), size = fabsf(v);
                // the largest finite sum of these 32 columns of the row
                const uint32_t most = __reduce_max_sync(0xffffffffu, m < p.m && size < INFINITY ? __float_as_uint(size) : 0u);
                const float near = __uint_as_float(most) * p.near;
                if (rounds_apart<T>(v - near, v + near)) marks |= 1u << e;
              }
              // fewer than eight columns say too little of how large the parts of a sum were: all in order
              if (p.m - (m - lane) < 8) marks = n == 32 ? 0xffffffffu : (1u << n) - 1u;
              if (m < p.m) p.unsure[(static_cast<int64_t>(w.r) * ((p.tile_n + 31) / 32) + j / 32) * p.m + m] = marks;
            };
            if (p.out_type == SPGEMM_DTYPE_BF16) mark(__nv_bfloat16());
            else mark(__half());
          }
          uint32_t odd = 0;  // Adapted: sums to form again
          if (MODE == kMmaAdapted) {
            uint32_t worst = 0;  // twice the bits: no sign
#pragma unroll
            for (int e = 0; e < 32; ++e) worst = max(worst, r[e] + r[e]);
            if (worst >= 0xff000000u && m < p.m) {
#pragma unroll
              for (int e = 0; e < 32; ++e) odd |= not_finite(r[e]) && e < n ? 1u << e : 0u;
            }
          }
          int token = 0;
          float f = 1.0f;
          if (MODE == kMmaForward && p.scatter) {  // rows leave in the tokens' order
            token = lane < n ? max(p.order[t.j0 + j + lane], 0) / p.top_k : 0;
            if (p.scale) f = p.scale[t.g];
          }
          auto put = [&](auto type) {
            using T = decltype(type);
            T* out = static_cast<T*>(p.out);
            if (MODE == kMmaForward && p.scatter) {
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const int64_t row = __shfl_sync(0xffffffffu, token, e);
                if (e < n && m < p.m) out[row * p.out_stride + m] = from_f32<T>(f * __uint_as_float(r[e]));
              }
            } else if (n == 32) {
              if (m < p.m) {
#pragma unroll
                for (int e = 0; e < 32; ++e) out[o + e * p.out_stride] = from_f32<T>(__uint_as_float(r[e]));
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e < n && m < p.m) out[o + e * p.out_stride] = from_f32<T>(__uint_as_float(r[e]));
            }
            if constexpr (MODE == kMmaAdapted && sizeof(T) == 2) {
              for (uint32_t any = __reduce_or_sync(0xffffffffu, odd); any; any &= any - 1) {
                const int e = __ffs(any) - 1;
                float sum = 0.0f;
                const uint32_t again = own_sums<T>(p, t.j0, t.n, t.j0 + j + e, m - lane,
                                                   __ballot_sync(0xffffffffu, (odd >> e) & 1u), &sum);
                if ((again >> lane) & 1u) out[o + e * p.out_stride] = from_f32<T>(sum);
              }
            }
          };
          if (p.out_type == SPGEMM_DTYPE_F32) put(float());
          else if (p.out_type == SPGEMM_DTYPE_BF16) put(__nv_bfloat16());
          else put(__half());
        }
      }
      if (!zero) {
        fence_before();
        if (PAIR) mbar_arrive_cluster(map_rank(smem_u32(&c.acc_empty[it & 1]), 0));
        else mbar_arrive(smem_u32(&c.acc_empty[it & 1]));
        ++it;
      }
    }
    // rows behind the last group
    if ((MODE == kMmaForward || MODE == kMmaGated) && !p.scatter) {
      for (int64_t r = c.first[p.groups] + blockIdx.x; r < p.slots; r += gridDim.x)
        for (int m = static_cast<int>(threadIdx.x) - (kThreads - kEpilogue); m < p.m; m += kEpilogue) {
          const int64_t o = r * p.out_stride + m;
          if (p.out_type == SPGEMM_DTYPE_F32) static_cast<float*>(p.out)[o] = 0.0f;
          else static_cast<uint16_t*>(p.out)[o] = 0;
        }
    }
  }
  if (p.early) {  // blocks without a tile, and tiles without an adapter, have not waited yet
    pdl_wait();
    pdl_go();
  }
  fence_before();
  __syncthreads();
  if (SPLIT) {
    // Every block has its part of the sums; the stages are idle in all of them.  Block q of the cluster adds
    // up columns [q, q + 1) * width of the tile (width a power of two, 4 at least): buf[source][lane][column].
    cluster_sync();
    fence_after();
    const int width = p.tile_n / parts, shift = 31 - __clz(width);
    Walk w = start();
    const bool there = w.r < all_tiles && !*failed && warp > kProducers;
    const Tile t = there ? tile_of(w) : Tile{};
    const int ml = (warp & 3) * 32 + lane, set = (warp - kProducers - 1) >> 2;
    if (there) {
      const uint32_t acc = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      for (int j = set * 32; j < t.n; j += 32 * kSets) {
        uint32_t r[32];
        tmem_load32(acc + j, r);
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          if (j + e < t.n) {
            const int owner = (j + e) >> shift, col = (j + e) & (width - 1);
            store_cluster(map_rank(base + ((part * 128 + ml) * width + col) * 4, owner), r[e], r[e + 1], r[e + 2], r[e + 3]);
          }
      }
    }
    cluster_sync();
    if (there) {
      const int m = t.m0 + ml, first = t.j0 + part * width;
      const int cols = min(width, t.n - part * width);
      for (int col = set * 4; col < cols; col += 4 * kSets) {
        float sum[4] = {};
        for (int q = 0; q < parts; ++q) {
          const float4 v = *reinterpret_cast<const float4*>(smem_raw + (base - smem_u32(smem_raw)) + ((q * 128 + ml) * width + col) * 4);
          sum[0] += v.x;
          sum[1] += v.y;
          sum[2] += v.z;
          sum[3] += v.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (col + e >= cols) continue;
          int64_t row = first + col + e;
          if (MODE == kMmaAdapted) {
            const uint32_t odd = __ballot_sync(0xffffffffu, m < p.m && not_finite(__float_as_uint(sum[e])));
            if (odd && p.bf16) own_sums<__nv_bfloat16>(p, t.j0, t.n, static_cast<int>(row), m - (threadIdx.x & 31), odd, &sum[e]);
            else if (odd) own_sums<__half>(p, t.j0, t.n, static_cast<int>(row), m - (threadIdx.x & 31), odd, &sum[e]);
          }
          if (m >= p.m) continue;
          if (MODE == kMmaForward && p.scatter) {
            row = max(p.order[row], 0) / p.top_k;
            if (p.scale) sum[e] *= p.scale[t.g];
          }
          const int64_t o = row * p.out_stride + m;
          if (p.out_type == SPGEMM_DTYPE_F32) static_cast<float*>(p.out)[o] = sum[e];
          else if (p.out_type == SPGEMM_DTYPE_BF16) static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(sum[e]);
          else static_cast<__half*>(p.out)[o] = __float2half_rn(sum[e]);
        }
      }
    }
    fence_before();
    __syncthreads();
  }
  if (PAIR) cluster_sync();
  fence_after();
  if (warp == kProducers) tmem_free<PAIR>(tmem, tmem_cols);
}

namespace {

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder() {
  static const Encode fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<Encode>(f);
  }();
  return fn;
}

// rank 2 or 3 map of 16-bit elements with 128-byte swizzle; dims[0] is contiguous
bool encode(CUtensorMap* map, int32_t dtype, const void* data, int rank, const int64_t* dims, const int64_t* strides,
            uint32_t box_cols, uint32_t box_rows) {
  const Encode fn = encoder();
  if (!fn) return false;
  cuuint64_t d[3], st[2];
  const cuuint32_t box[3] = {box_cols, box_rows, 1}, ones[3] = {1, 1, 1};
  for (int i = 0; i < rank; ++i) d[i] = static_cast<cuuint64_t>(dims[i]);
  for (int i = 0; i + 1 < rank; ++i) st[i] = static_cast<cuuint64_t>(strides[i]) * 2;
  return fn(map, dtype == SPGEMM_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
            static_cast<cuuint32_t>(rank), const_cast<void*>(data), d, st, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

bool encode_rows(CUtensorMap* map, const spgemm_dense& m, uint32_t box_rows) {
  const int64_t dims[2] = {m.cols, m.rows}, strides[1] = {m.stride};
  return encode(map, m.dtype, m.data, 2, dims, strides, kDeep, box_rows);
}
bool encode_weights(CUtensorMap* map, const spgemm_weights& w) {
  // a single group may carry any group stride: a map wants a multiple of 16 bytes
  const int64_t dims[3] = {w.cols, w.rows, w.groups};
  const int64_t strides[2] = {w.row_stride, w.groups > 1 ? w.group_stride : w.row_stride * w.rows};
  return encode(map, w.dtype, w.data, 3, dims, strides, kDeep, 64);
}

}  // namespace

int sm_count() {
  static const int sms = [] {  // the library runs on one kind of device
    int dev = 0, n = 1;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
  }();
  return sms;
}

namespace {

template <int MODE, bool PAIR, bool SPLIT>
bool launch(const MmaMaps& maps, MmaArgs a, int64_t grid, cudaStream_t s) {
  a.sub_bytes = kABytes + std::max(a.tile_n / (PAIR ? 2 : 1), MODE == kMmaDw ? 64 : 16) * 128;
  a.stage_bytes = a.sub_bytes * (SPLIT ? 1 : 2);
  const int control = static_cast<int>(sizeof(Control) + (MODE == kMmaGated ? sizeof(Swap) : 0));
  // split: two blocks per SM, and the stages hold the sums that meet there
  const int most = SPLIT ? kSmemMost / 2 - 1024 : kSmemMost;
  a.stages = std::min<int>(kMaxStages, (most - 1024 - control) / a.stage_bytes);
  const int smem = 1024 + a.stages * a.stage_bytes + control;
  auto kern = k_group_mma<MODE, PAIR, SPLIT>;
  static std::atomic<uint64_t> raised{0};  // devices on which the kernel may use this much shared memory
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(raised.load(std::memory_order_relaxed) & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) != cudaSuccess) return false;
    raised.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {SPLIT ? static_cast<unsigned>(a.split) : PAIR ? 2u : 1u, 1u, 1u};
  cfg.attrs = attr;
  cfg.numAttrs = PAIR || SPLIT ? 2 : 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kern, maps, a) == cudaSuccess;
}

template <int MODE>
bool launch_whole(const MmaMaps& maps, const MmaArgs& a, bool pair, cudaStream_t s) {
  const int64_t grid = sm_count() / 2 * 2;
  return pair ? launch<MODE, true, false>(maps, a, grid, s) : launch<MODE, false, false>(maps, a, grid, s);
}

// Width of the N-side tile, whether two blocks share it, and how many share its depth.
struct Width {
  int n;
  bool pair;
  int split;
};

// set by tests, for the calls of their own thread
thread_local int32_t t_hold = 0, t_polls = 0;
thread_local Width t_width = {0, false, 0};

// What a test asked for, as far as the kernel at hand allows it (widths from `least` to `most`, and the limits of
// most_split() without its question whether there are idle SMs); nothing asked: `rule`.
Width chosen(const Width& rule, int least, int most, bool splits, int64_t slices) {
  if (!t_width.n) return rule;
  Width w{std::min(std::max(t_width.n, least), most), false, 1};
  w.pair = t_width.pair && w.n == 256;
  if (splits && w.n <= kSplitTile)
    while (w.split < t_width.split && w.split * 4 <= slices && w.split * 8 <= w.n) w.split *= 2;
  return w;
}

// The most blocks (up to 8) that may share a tile's depth: only where the tiles (at most `tiles`) leave half
// the SMs idle, as many as fit at two per SM, with at least two slices each.
int most_split(int n, int64_t tiles, int64_t slices) {
  int split = 1;
  if (n <= kSplitTile && tiles * 2 <= sm_count())
    while (split < 8 && tiles * split <= sm_count() && split * 4 <= slices && split * 8 <= n) split *= 2;
  return split;
}

// The width with the least waves x cycles of a tile.  A slice takes the longer of its instructions (two
// cycles per column) and its bytes at 60 per cycle and SM, a tile the longer of its slices and of the
// epilogue (12 cycles per column) plus 1000 to change over, or 8000 for the meeting of a split tile's blocks;
// `tiles(n)` of them on the N side.
// The constants are estimates from the kernel's traffic and from profiles, not a fit.  Held against every width a
// kernel can take (48 sweeps: forward, layer, dx, dw and adapted, 64 to 65536 rows, 4 to 64 groups, 280 to 8192 deep):
// within 1% of the best in 28, 5% above it on average, at worst 40% (six rows in each of 64 groups: tiles of 16 rows
// 35 us, of 64 rows 25 us; the groups' sizes are not known here).
template <typename F>
Width pick_width(int64_t m, int m_per_block, int64_t slices, int least, bool splits, F tiles) {
  Width best{256, true, 1};
  double least_time = -1.0;
  for (int n = 256; n >= least; n /= 2)
    for (int side = n == 256 ? 2 : 1; side >= 1; --side) {
      const int64_t all = tiles(n) * ceil_div(m, m_per_block * side);
      const int split = splits && side == 1 ? most_split(n, all, slices) : 1;
      const double slice = std::max(2.0 * n, (16384.0 + n / side * 128.0) / 60.0);
      const double crowd = all * split > sm_count() ? 1.5 : 1.0;  // two blocks of a split tile on one SM
      const double tile = split > 1 ? ceil_div(slices, split) * slice * crowd + 8000.0
                                    : std::max(slices * slice, 12.0 * n) + 1000.0;
      const double waves = split > 1 ? 1.0 : std::ceil(static_cast<double>(all) / (sm_count() / side));
      const double time = waves * tile + 12.0 * n;
      if (least_time < 0.0 || time < least_time) {
        least_time = time;
        best = Width{n, side == 2, split};
      }
    }
  return chosen(best, least, 256, splits, slices);
}

// N-side tiles of a grouping whose groups are not known here: each group that has rows ends in a part tile
int64_t likely_tiles(const spgemm_grouping& g, int n) {
  const int64_t used = std::min<int64_t>(g.groups, g.slots);
  return std::max(used, g.slots / n + used / 2);
}

// Measured at 64 rows, 4096 x 4096, 48 adapters: 4 blocks per tile 19 us, 8 blocks 13 us; with three quarters of
// the SMs busy (125 tiles, 16 slices) 13 us whole, 18 us split.
template <int MODE>
bool launch_split(const MmaMaps& maps, MmaArgs a, const Width& width, int64_t tiles, cudaStream_t s) {
  if (width.split == 1) return launch_whole<MODE>(maps, a, width.pair, s);
  a.split = width.split;
  return launch<MODE, false, true>(maps, a, tiles * a.split, s);
}

// most tiles on the N side: every group may end in a part of one
int64_t most_tiles(const spgemm_grouping& g, int tile_n) {
  return g.slots / tile_n + std::min<int64_t>(g.groups, g.slots);
}


MmaArgs base_args(const spgemm_grouping& g, int32_t dtype) {
  MmaArgs a = {};
  a.hold = t_hold;
  a.polls = t_polls > 0 ? static_cast<uint32_t>(t_polls) : tc::kMaxPolls;
  a.offsets = g.offsets;
  a.order = g.order;
  a.slots = static_cast<int>(g.slots);
  a.groups = g.groups;
  a.top_k = g.top_k;
  a.bf16 = dtype == SPGEMM_DTYPE_BF16;
  a.err = grouped_err();
  return a;
}

bool aligned(const void* p, int64_t stride) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0; }

}  // namespace

void mma_debug(int32_t hold, int32_t polls) {
  t_hold = hold;
  t_polls = polls;
}
void mma_force(int32_t width, int32_t pair, int32_t split) { t_width = Width{width, pair != 0, split}; }

// Gathered against laid out first, 2048 x 2048, 64 groups of 32 rows 93 us and 94, of 96 rows 109 and 110, of 128 rows 152
// and 116, of 512 rows 452 and 245; 16 groups of 32 rows 30 and 31; 8 groups of 16 rows, 4096 x 1024, 24 and 26.
bool mma_gathers(const spgemm_grouping& g) { return g.slots <= 64 * static_cast<int64_t>(g.groups); }

bool mma_takes(const spgemm_dense& m) { return m.dtype != SPGEMM_DTYPE_F32 && aligned(m.data, m.stride) && m.rows < (1LL << 31) && m.cols < (1LL << 31); }
bool mma_takes(const spgemm_weights& w) {
  return w.dtype != SPGEMM_DTYPE_F32 && aligned(w.data, w.row_stride) && (w.groups == 1 || (w.group_stride > 0 && w.group_stride % 8 == 0)) &&
         w.rows < (1LL << 30) && w.cols < (1LL << 30);
}

namespace {

// How far the tensor cores' sum of `depth` products may be from the 32-bit sum in index order, in units of the
// largest sum of the row's 32 columns beside it: half a unit in the last place (2^-24) for each of its depth / 16
// additions, and 16 more for the other order's own roundings.  Largest distance measured, in units of this:
// 0.97 in 7e8 sums of normal, uniform and shifted values and rows of very different sizes, 64 to 8192 terms; 1.22 where a
// hundredth of the features is thirty times the rest.  No element of these was rounded another way without being
// marked.  Half of this would mark 45% fewer and leave up to 1e-6 of the elements (5e-5 of 8192 shifted terms) wrong.
float near_of(int64_t depth) { return static_cast<float>(depth + 256) * 0x1p-28f; }

// Tiles of gathered rows belong to single blocks and have 128 rows at most: groups with more come laid out.
Width forward_width(const spgemm_grouping& g, const spgemm_dense& x, bool gather, bool gated, int64_t cols) {
  const Width width =
      pick_width(cols, gated ? 64 : 128, ceil_div(x.cols, kDeep), 16, false, [&](int n) { return likely_tiles(g, n); });
  return gather && width.n > 128 ? Width{128, false, 1} : width;
}

}  // namespace

int mma_forward_tile(const spgemm_grouping& g, const spgemm_dense& x, bool gather, int64_t cols) {
  return forward_width(g, x, gather, false, cols).n;
}

int64_t mma_likely_tiles(const spgemm_grouping& g, int tile_n) { return likely_tiles(g, tile_n); }

int64_t mma_marks_bytes(const spgemm_grouping& g, int tile_n, int64_t cols) {
  return 4 * most_tiles(g, tile_n) * ceil_div(tile_n, 32) * cols;
}

bool launch_mma_forward(const spgemm_grouping& g, const spgemm_dense& x, bool gather, const spgemm_weights& w,
                        bool gated, const spgemm_dense& y, uint32_t* unsure, bool early, cudaStream_t s) {
  if (g.slots == 0) return true;
  MmaArgs a = base_args(g, x.dtype);
  a.early = early;
  a.rows = static_cast<int>(x.rows);
  a.gather = gather;
  a.m = static_cast<int>(y.cols);
  a.depth = static_cast<int>(x.cols);
  const Width width = forward_width(g, x, gather, gated, y.cols);
  a.tile_n = width.n;
  a.box_rows = std::min(a.tile_n, 64);
  a.out = y.data;
  a.out_stride = y.stride;
  a.out_type = y.dtype;
  a.unsure = unsure;
  a.near = near_of(x.cols);
  MmaMaps maps;
  if (!encode_weights(&maps.a, w) || !encode_rows(&maps.b, x, gather ? 1 : a.box_rows)) return false;
  maps.c = maps.d = maps.b;
  return gated ? launch_whole<kMmaGated>(maps, a, width.pair, s) : launch_whole<kMmaForward>(maps, a, width.pair, s);
}

bool launch_mma_dx(const spgemm_grouping& g, const spgemm_dense& dy, const spgemm_weights& w, float* dx,
                   cudaStream_t s) {
  if (g.slots == 0) return true;
  MmaArgs a = base_args(g, dy.dtype);
  a.rows = static_cast<int>(dy.rows);
  a.m = static_cast<int>(w.cols);
  a.depth = static_cast<int>(w.rows);
  const Width width = pick_width(a.m, 128, ceil_div(a.depth, kDeep), 16, false, [&](int n) { return likely_tiles(g, n); });
  a.tile_n = width.n;
  a.box_rows = std::min(a.tile_n, 64);
  a.out = dx;
  a.out_stride = w.cols;
  a.out_type = SPGEMM_DTYPE_F32;
  MmaMaps maps;
  if (!encode_weights(&maps.a, w) || !encode_rows(&maps.b, dy, a.box_rows)) return false;
  maps.c = maps.d = maps.b;
  return launch_whole<kMmaDx>(maps, a, width.pair, s);
}

bool launch_mma_dw(const spgemm_grouping& g, const spgemm_dense& dy, const spgemm_dense& x, const spgemm_weights& dw,
                   cudaStream_t s) {
  MmaArgs a = base_args(g, x.dtype);
  a.m = static_cast<int>(dw.cols);
  a.n = static_cast<int>(dw.rows);
  const Width width = pick_width(a.m, 128, ceil_div(ceil_div(g.slots, g.groups), kDeep), 64, false,
                                 [&](int n) { return g.groups * ceil_div(dw.rows, n); });
  a.tile_n = width.n;
  a.out = dw.data;
  a.out_stride = dw.row_stride;
  a.out_group = dw.group_stride;
  a.out_type = dw.dtype;
  MmaMaps maps;
  if (!encode_rows(&maps.a, x, 64) || !encode_rows(&maps.b, dy, 64) || !encode_rows(&maps.c, dy, 1) ||
      !encode_rows(&maps.d, x, 1))
    return false;
  return launch_whole<kMmaDw>(maps, a, width.pair, s);
}

bool launch_mma_shrink(const spgemm_grouping& g, const spgemm_dense& x, const spgemm_weights& a_w, const float* scale,
                       const spgemm_dense& v, cudaStream_t s) {
  MmaArgs a = base_args(g, x.dtype);
  a.rows = static_cast<int>(x.rows);
  a.gather = a.scatter = 1;
  a.m = static_cast<int>(v.cols);
  a.depth = static_cast<int>(x.cols);
  // The widest tile that still gives every SM one: x is read once either way, a's rows once per tile.  The whole call
  // with 16 adapters, rank 64, 64 outputs: 8192 rows of 4096, tiles of 32 72 us, 64 54 us, 128 59 us; 20000 rows of 2048
  // 75, 57 and 52 us.  (2048 rows: 41 us with the 32 that this takes, 35 with 64.)
  a.tile_n = 32;
  while (a.tile_n < 128 && g.slots > static_cast<int64_t>(a.tile_n) * sm_count()) a.tile_n *= 2;
  const Width asked = chosen(Width{a.tile_n, false, 0}, 32, 128, true, ceil_div(a.depth, kDeep));
  a.tile_n = asked.n;
  const int64_t tiles = most_tiles(g, a.tile_n) * ceil_div(a.m, 128);
  const Width width{a.tile_n, false, asked.split ? asked.split : most_split(a.tile_n, tiles, ceil_div(a.depth, kDeep))};
  a.box_rows = 32;
  a.out = v.data;
  a.out_stride = v.stride;
  a.out_type = v.dtype;
  a.scale = scale;
  MmaMaps maps;
  a.runs = 1;
  if (!encode_weights(&maps.a, a_w) || !encode_rows(&maps.b, x, 1) || !encode_rows(&maps.c, x, a.box_rows)) return false;
  maps.d = maps.b;
  return launch_split<kMmaForward>(maps, a, width, tiles, s);
}

bool launch_mma_adapted(const spgemm_dense& x, const spgemm_dense& w, const spgemm_weights& b, const int32_t* ids,
                        const spgemm_dense& v, const spgemm_dense& y, cudaStream_t s) {
  MmaArgs a = base_args(spgemm_grouping{x.rows, 1, 1, nullptr, nullptr, nullptr}, x.dtype);
  a.rows = static_cast<int>(x.rows);
  a.ids = ids;
  a.adapters = static_cast<int>(b.groups);
  a.rank = static_cast<int>(b.cols);
  a.x = x.data;
  a.x_stride = x.stride;
  a.w = w.data;
  a.w_stride = w.stride;
  a.v = v.data;
  a.v_stride = v.stride;
  a.b = b.data;
  a.b_stride = b.row_stride;
  a.b_group = b.group_stride;
  a.early = 1;
  a.m = static_cast<int>(y.cols);
  a.depth = static_cast<int>(x.cols);
  const Width width =
      pick_width(a.m, 128, ceil_div(a.depth, kDeep), 16, true, [&](int n) { return ceil_div(x.rows, n); });
  a.tile_n = width.n;
  a.box_rows = std::min(a.tile_n, 64);
  a.out = y.data;
  a.out_stride = y.stride;
  a.out_type = y.dtype;
  const spgemm_weights shared{w.data, 1, w.rows, w.cols, 0, w.stride, w.dtype, 0};
  MmaMaps maps;
  if (!encode_weights(&maps.a, shared) || !encode_rows(&maps.b, x, a.box_rows) || !encode_weights(&maps.c, b) ||
      !encode_rows(&maps.d, v, 1))
    return false;
  return launch_split<kMmaAdapted>(maps, a, width, ceil_div(x.rows, a.tile_n) * ceil_div(a.m, 128), s);
}

}  // namespace sg
