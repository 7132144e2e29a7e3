// Grouped products in 8-bit floating point on the tensor cores (tcgen05, e4m3 inputs, scales in the instruction):
//
//   y[p, n] = sum_b sx[p, b] sw[n / 128, b] sum_{k in block b} x[p, k] w[g][n, k]
//
// The scales are powers of two, and the matrix instruction multiplies with such scales itself: one for every 32 numbers
// along the contracted index, four alike for a block of 128.  So the sums of all blocks stay in one accumulator, in 32
// bits, and nothing comes between the matrix instructions.  (Scales of any kind want each block's sums read back, multiplied
// and added in registers; that took 850 to 1400 cycles a block, however divided over warps, where the instructions take 512:
// 238 to 264 us for the product below.)
//
// M is the rows of a group (128 of them, 256 for a pair of blocks), N the matrix's rows, up to 240: two accumulators of 240
// columns and the scales of two slices are what tensor memory holds.
//
// Sixteen warps: two producers (bulk copies of 128-byte swizzled boxes, one for each operand: a copy takes its thread about
// 150 cycles to issue, a slice's instructions 480), two issuers, four that bring scales into the instruction's layout, a stage
// each, and two sets of four that empty an accumulator while the other is filled; a tile leaves through shared memory, so that a row's
// piece is written 64 bytes at a time.  A stage holds two slices of 128.  Persistent blocks; pairs of blocks
// share a tile (cta_group::2): each holds half of both operands.
//
// Measured: 49152 rows in 64 groups, 2048 x 2048: 178 us, 2320 TFLOP/s (unequal groups, last tiles part empty); 65536 rows in 32
// groups 206 us, 2670 TFLOP/s.  The tensor pipe is busy 60% of the time, and the tiles take 40 bytes per cycle and SM from L2, less than
// the 16-bit kernel (47): neither is at its limit, and what holds the rest is not established.  96 rows in 64 groups: 34 to 37 us,
// 190 MB at 5.1 to 5.6 TB/s.  Fetching later stages into L2 first made it
// slower (211 us for the first), and so did one accumulator of 448 columns (245 us: nothing runs while it is emptied).
//
// Every wait is bounded: a role that gives up sets the status word, the others see it, copies in flight are drained,
// tensor memory is freed, the kernel returns.
#include <algorithm>
#include <atomic>

#include "group_mma.h"
#include "quant8.cuh"
#include "tc.cuh"

namespace sg {

namespace {

constexpr int kEpilogue = 8;         // warps 4 to 11, two sets of four
constexpr int kMaxStages = 4;
constexpr int kScalers = 4;          // warps 12 to 15, each with its part of the ring of scales
constexpr int kThreads = 32 * (4 + kEpilogue + kScalers);
constexpr int kSub = 2;              // slices of a stage
constexpr int kMostCols = 240;       // of a tile
constexpr int kXBytes = 128 * kBlock8;      // the group's rows' part of a slice
constexpr int kScaleBytes = 3 * 512;        // of a stage: words of 128 rows and of 2 x 128 of the matrix's, a byte per slice
static_assert(kSub == 2, "the issuer's two halves of a stage");
constexpr int kOut = 64;             // bytes of a row's piece on its way out
constexpr int kOutRow = kOut + 16;   // and room so that no two rows share a bank
constexpr int kTmemCols = 512, kTmemScales = 2 * kMostCols;  // scales of a stage: four columns of x's, eight of w's; of two stages by turns
constexpr int kSmemMost = 227 * 1024;

struct Control {
  alignas(128) uint8_t scales[kScalers][kScaleBytes];
  alignas(16) char out[kEpilogue][32][kOutRow];
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t scale_full[kScalers], scale_empty[kScalers];
  uint64_t acc_full[2], acc_empty[2], turn[2], drain[2];
  uint32_t tmem;
  int failed[2];                   // a role gave up; polls allowed to a wait
  int scan[33];
  int first[kMaxGroups + 1];       // first position of each group (clamped to [0, slots])
  int tiles[kMaxGroups + 1];       // row tiles of the groups before each
};

struct Args {
  const int32_t* offsets;
  int slots, groups;
  int early;               // the kernel before makes only x: start without waiting for it
  int n, blocks;           // rows of a matrix (columns of y), blocks of 128 along the contracted index
  int tile_n;
  int stages, stage_bytes, sub_bytes;
  const float *sx, *sw;
  int64_t sx_stride;
  void* out;
  int64_t out_stride;
  int out_type, wide;      // wide: y's rows start on 16 bytes
  uint32_t* err;
  uint32_t polls;
  int hold;
};

struct Tile {
  int g, n0;     // group, first column
  int j0, rows;  // first position, and how many there are
};

// The scales' exponents as the instruction wants them, a byte per slice; odd: one that is no power of two in range.
__device__ __forceinline__ uint32_t scale_word(const float (&s)[kSub], bool& odd) {
  uint32_t word = 0;
#pragma unroll
  for (int h = 0; h < kSub; ++h) {
    const uint32_t u = __float_as_uint(s[h]);
    odd = odd || (u & 0x807fffffu) != 0 || u == 0 || u >= 0x7f800000u;
    word |= (u >> 23 & 255u) << (8 * h);
  }
  return word;
}

}  // namespace

template <bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) k_group_8bit(const __grid_constant__ CUtensorMap map_w,
                                                            const __grid_constant__ CUtensorMap map_x,
                                                            const __grid_constant__ Args p) {
  using namespace tc;
  extern __shared__ char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  Control& c = *reinterpret_cast<Control*>(smem_raw + (base - smem_u32(smem_raw)) + p.stages * p.stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0u;
  constexpr int kSide = PAIR ? 2 : 1, kRows = 128 * kSide;
  volatile int* failed = c.failed;

  // ---- set-up: barriers, tensor memory, the groups' first positions and tile counts -----------
  if (warp == 0) {
    if (lane < p.stages) {
      // two announcements of bytes; tests: an arrival that never comes, on the first stage of block 0
      mbar_init(smem_u32(&c.full[lane]), p.hold && blockIdx.x == 0 && lane == 0 ? 3 : 2);
      mbar_init(smem_u32(&c.empty[lane]), 1);
    } else if (lane < p.stages + 2) {
      mbar_init(smem_u32(&c.acc_full[lane - p.stages]), 1);
      mbar_init(smem_u32(&c.acc_empty[lane - p.stages]), kEpilogue * kSide);
    } else if (lane >= 16 && lane < 16 + kScalers) {
      mbar_init(smem_u32(&c.scale_full[lane - 16]), kSide);
      mbar_init(smem_u32(&c.scale_empty[lane - 16]), 1);
    } else if (lane == 31) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&c.turn[i]), 1);
        mbar_init(smem_u32(&c.drain[i]), 1);
      }
      c.failed[0] = 0;
      c.failed[1] = static_cast<int>(p.polls);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (warp == 4 && lane == 0) {
    prefetch_map(&map_w);
    prefetch_map(&map_x);
  }
  if (PAIR) cluster_sync();  // both blocks run before one allocates in both
  if (warp == 1) tmem_alloc<PAIR>(smem_u32(&c.tmem), kTmemCols);
  if (!p.early) {
    pdl_wait();
    pdl_go();
  }
  // offsets are used as a non-decreasing sequence inside [0, slots], whatever the array holds.  Where the kernel starts early they
  // are read before its wait: the kernel ahead, which makes only x's rows, waited for everything before it and let this one start
  // after that, so they were complete.  Past L1: a call before may have left other offsets there, at the same address.
  {
    int run = 0;
    for (int g0 = 0; g0 < p.groups; g0 += kThreads) {
      const int g = g0 + static_cast<int>(threadIdx.x);
      int lo = 0, hi = 0;
      if (g < p.groups) {
        lo = min(max(__ldcg(p.offsets + g), 0), p.slots);
        hi = min(max(__ldcg(p.offsets + g + 1), lo), p.slots);
        c.first[g] = lo;
        if (g == p.groups - 1) c.first[p.groups] = hi;
      }
      const int n = (hi - lo + kRows - 1) / kRows;
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
  const int nt = (p.n + p.tile_n - 1) / p.tile_n;
  const int worker = static_cast<int>(PAIR ? blockIdx.x >> 1 : blockIdx.x);
  const int workers = static_cast<int>(PAIR ? gridDim.x >> 1 : gridDim.x);

  // columns fastest, then the rows, group by group: blocks that run at the same time share a group in L2
  const int all_tiles = c.tiles[p.groups];
  struct Walk {
    int n, r, g;
  };
  const int step_n = workers % nt, step_r = workers / nt;
  auto start = [&]() { return Walk{worker % nt, worker / nt, 0}; };
  auto advance = [&](Walk& w) {
    w.n += step_n;
    w.r += step_r;
    if (w.n >= nt) {
      w.n -= nt;
      ++w.r;
    }
  };
  auto tile_of = [&](Walk& w) {
    while (w.g + 1 < p.groups && c.tiles[w.g + 1] <= w.r) ++w.g;
    const int lo = c.first[w.g], hi = max(c.first[w.g + 1], lo);
    Tile t;
    t.g = w.g;
    t.n0 = w.n * p.tile_n;
    t.j0 = lo + (w.r - c.tiles[w.g]) * kRows;
    t.rows = min(hi - t.j0, kRows);
    return t;
  };
  int s = 0;  // stage, of the roles that pass them
  uint32_t phase = 0;
  auto close = [&]() {
    if (++s == p.stages) {
      s = 0;
      phase ^= 1u;
    }
  };


  if (warp == 0 || warp == 3) {
    // ---- producers: one lane each, of the matrix's rows (warp 0) and of the group's (warp 3) --------
    if (lane == 0) {
      const bool rows = warp == 3;
      bool ok = true;
      const uint32_t full0 = PAIR ? map_rank(smem_u32(&c.full[0]), 0) : smem_u32(&c.full[0]);
      const uint32_t dst = base + (rows ? 0 : kXBytes);
      if (rows && p.early) {  // the group's rows are the kernel's before this one, the matrices are not
        pdl_wait();
        pdl_go();
      }
      for (Walk w = start(); w.r < all_tiles && ok; advance(w)) {
        const Tile t = tile_of(w);
        const uint32_t bytes = static_cast<uint32_t>((rows ? 128 : p.tile_n / kSide) * kBlock8) * kSide;
        const int first = rows ? t.j0 + static_cast<int>(rank) * 128 : t.n0 + static_cast<int>(rank) * (p.tile_n / kSide);
        for (int q = 0; q < p.blocks; q += kSub) {
          ok = mbar_wait(smem_u32(&c.empty[s]), phase ^ 1u, failed, p.err, 1u);
          if (!ok) break;
          const int subs = min(kSub, p.blocks - q);
          if (rank == 0) mbar_expect_tx(smem_u32(&c.full[s]), subs * bytes);
          const uint32_t bar = full0 + s * 8u;
          for (int h = 0; h < subs; ++h) {
            const uint32_t to = dst + s * p.stage_bytes + h * p.sub_bytes;
            if (rows) load_2d<PAIR>(to, &map_x, (q + h) * kBlock8, first, bar);  // 128 of them, however many are the group's
            else load_3d<PAIR>(to, &map_w, (q + h) * kBlock8, first, t.g, bar);
          }
          close();
        }
      }
      // after a failure nothing consumes the stages any more: wait for the copies in flight
      if (*failed) {
        for (int q = 0; q < p.stages; ++q) {
          mbar_drain(smem_u32(&c.full[s]), phase ^ 1u, max(p.polls >> 4, 64u));
          close();
        }
      }
    }
    __syncwarp();
  } else if (warp >= 4 + kEpilogue) {
    // ---- scales: rows lane, lane + 32, ... of each 128.  The ring is not the operands': what is between a free stage and
    // the next instruction is a copy, not a warp's stores and fences, which take as long ---------------------
    if (p.early) pdl_wait();  // the rows' scales are the kernel's before this one
    const int col_blocks = (p.n + kBlock8 - 1) / kBlock8, mine = warp - 4 - kEpilogue;
    bool ok = true, odd = false;
    const uint32_t full = PAIR ? map_rank(smem_u32(&c.scale_full[mine]), 0) : smem_u32(&c.scale_full[mine]);
    int k = 0;  // stages so far, of all
    for (Walk w = start(); w.r < all_tiles && ok; advance(w)) {
      const Tile t = tile_of(w);
      const int row0 = static_cast<int>(rank) * 128 + lane, nb0 = t.n0 / kBlock8;
      const float* sx = p.sx + t.j0 + row0;
      // a tile's columns lie in up to three blocks of 128 rows of the matrix
      const float* sw = p.sw + (static_cast<int64_t>(t.g) * col_blocks + nb0) * p.blocks;
      const int most = col_blocks - 1 - nb0;
      for (int q = 0; q < p.blocks; q += kSub, ++k) {
        if (k % kScalers != mine) continue;
        float v[4][kSub], f[3][kSub];
#pragma unroll
        for (int h = 0; h < kSub; ++h) {
          const bool slice = q + h < p.blocks;
#pragma unroll
          for (int e = 0; e < 3; ++e) f[e][h] = slice ? sw[min(e, most) * p.blocks + q + h] : 1.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e][h] = slice && row0 + 32 * e < t.rows ? sx[(q + h) * p.sx_stride + 32 * e] : 1.0f;
        }
        ok = mbar_wait(smem_u32(&c.scale_empty[mine]), (k / kScalers & 1) ^ 1, failed, p.err, 16u);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint4* to = reinterpret_cast<uint4*>(c.scales[mine]) + lane;
        to[0] = make_uint4(scale_word(v[0], odd), scale_word(v[1], odd), scale_word(v[2], odd), scale_word(v[3], odd));
        const uint32_t word[3] = {scale_word(f[0], odd), scale_word(f[1], odd), scale_word(f[2], odd)};
        auto of = [&](int e) {
          const int b = min((t.n0 + lane + 32 * e) / kBlock8 - nb0, 2);
          return b == 0 ? word[0] : b == 1 ? word[1] : word[2];
        };
        to[32] = make_uint4(of(0), of(1), of(2), of(3));
        to[64] = make_uint4(of(4), of(5), of(6), of(7));
        fence_shared();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) mbar_arrive_cluster(full);
          else mbar_arrive(full);
        }
      }
    }
    if (__any_sync(0xffffffffu, odd) && lane == 0) set_error(p.err, kErrCsr);
  } else if (warp == 1 || warp == 2) {
    // ---- issuers: every other stage each.  Issuing a stage's instructions takes 700 cycles, finding the next one ready and giving
    // this one back 500; the instructions themselves run 960.  So one issuer gets ready while the other issues, and
    // hands over the turn: a stage's instructions follow the ones before it on the same sums. ---------------
    if (rank == 0 && lane == 0) {
      const int me = warp - 1;
      int it = 0, k = 0;
      const uint32_t idesc = instruction_scaled(kRows, p.tile_n);
      bool ok = true;
      for (Walk w = start(); w.r < all_tiles && ok; advance(w), ++it) {
        const uint32_t acc = tmem + (it & 1) * p.tile_n;
        for (int q = 0; q < p.blocks && ok; q += kSub, ++k, close()) {
          if ((k & 1) != me) continue;
          const int entry = k % kScalers;
          const uint32_t a = base + s * p.stage_bytes, scales = smem_u32(c.scales[entry]);
          const uint32_t sa = tmem + kTmemScales + me * 12, sb = sa + 4;
          ok = mbar_wait(smem_u32(&c.full[s]), phase, failed, p.err, 4u) &&
               mbar_wait(smem_u32(&c.scale_full[entry]), k / kScalers & 1, failed, p.err, 32u) &&
               (q > 0 || mbar_wait(smem_u32(&c.acc_empty[it & 1]), ((it >> 1) & 1) ^ 1u, failed, p.err, 2u)) &&
               (k == 0 || mbar_wait(smem_u32(&c.turn[me]), me == 0 ? (k / 2 - 1) & 1 : k / 2 & 1, failed, p.err, 64u));
          if (!ok) break;
          fence_after();
          copy_scales<PAIR>(sa, scales);
          copy_scales<PAIR>(sb, scales + 512);
          copy_scales<PAIR>(sb + 4, scales + 1024);
          mma_slice_scaled<PAIR>(acc, operand(a, 0), operand(a + kXBytes, 0), idesc, sa, sb, q > 0);
          if (q + 1 < p.blocks)
            mma_slice_scaled<PAIR>(acc, operand(a + p.sub_bytes, 0), operand(a + p.sub_bytes + kXBytes, 0), with_scale_byte(idesc, 1), sa, sb,
                                   true);
          fence_before();
          mbar_arrive(smem_u32(&c.turn[me ^ 1]));
          commit<PAIR>(smem_u32(&c.empty[s]));
          commit<PAIR>(smem_u32(&c.scale_empty[entry]));
          if (q + kSub >= p.blocks) commit<PAIR>(smem_u32(&c.acc_full[it & 1]));
        }
      }
      if (*failed) {
        commit<PAIR>(smem_u32(&c.drain[me]));
        mbar_drain(smem_u32(&c.drain[me]), 0, max(p.polls >> 4, 64u));
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---- epilogue --------------------------------------------------------------------------------------
    const int quarter = warp & 3, set = (warp - 4) >> 2;
    const int row0 = static_cast<int>(rank) * 128 + quarter * 32;  // the warp's first row of the tile
    int it = 0;
    for (Walk w = start(); w.r < all_tiles; advance(w), ++it) {
      const Tile t = tile_of(w);
      bool ok = mbar_wait(smem_u32(&c.acc_full[it & 1]), (it >> 1) & 1, failed, p.err, 8u);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      fence_after();
      const uint32_t acc = tmem + (it & 1) * p.tile_n + (static_cast<uint32_t>(quarter * 32) << 16);
      auto put = [&](auto type) {
        using T = decltype(type);
        constexpr int kPer = 16 / sizeof(T), kCols = kOut / sizeof(T);  // numbers of 16 bytes, and of a row's piece
        char(&stage)[32][kOutRow] = c.out[warp - 4];
        T* out = static_cast<T*>(p.out) + static_cast<int64_t>(t.j0 + row0) * p.out_stride + t.n0;
        for (int c0 = set * 32; c0 < p.tile_n; c0 += 64) {  // the sets take 32 columns by turns
          uint32_t r[32];
          tmem_load32(acc + c0, r);
#pragma unroll
          for (int h = 0; h < 32; h += kCols) {
#pragma unroll
            for (int e0 = 0; e0 < kCols; e0 += kPer) {
              alignas(16) T v[kPer];
#pragma unroll
              for (int e = 0; e < kPer; ++e) v[e] = from_f32<T>(__uint_as_float(r[h + e0 + e]));
              *reinterpret_cast<uint4*>(&stage[lane][e0 * sizeof(T)]) = *reinterpret_cast<const uint4*>(v);
            }
            __syncwarp();
            const int at = lane % 4 * kPer, cols = min(p.tile_n - c0, p.n - t.n0 - c0) - h;
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // eight rows at a time, four lanes each
              const int row = i * 8 + lane / 4;
              if (row0 + row < t.rows) {
                T* to = out + row * p.out_stride + c0 + h + at;
                const T* from = reinterpret_cast<const T*>(stage[row]) + at;
                if (p.wide && at + kPer <= cols) {
                  *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
                } else {
#pragma unroll
                  for (int e = 0; e < kPer; ++e)
                    if (at + e < cols) to[e] = from[e];
                }
              }
            }
            __syncwarp();
          }
        }
      };
      if (p.out_type == SPGEMM_DTYPE_F32) put(float());
      else if (p.out_type == SPGEMM_DTYPE_BF16) put(__nv_bfloat16());
      else put(__half());
      fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) mbar_arrive_cluster(map_rank(smem_u32(&c.acc_empty[it & 1]), 0));
        else mbar_arrive(smem_u32(&c.acc_empty[it & 1]));
      }
    }
    // rows behind the last group
    for (int64_t r = c.first[p.groups] + blockIdx.x; r < p.slots; r += gridDim.x)
      for (int n = static_cast<int>(threadIdx.x) - 128; n < p.n; n += 32 * kEpilogue) {
        const int64_t o = r * p.out_stride + n;
        if (p.out_type == SPGEMM_DTYPE_F32) static_cast<float*>(p.out)[o] = 0.0f;
        else static_cast<uint16_t*>(p.out)[o] = 0;
      }
  }
  fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();
  fence_after();
  if (warp == 1) tmem_free<PAIR>(tmem, kTmemCols);
}

namespace {

template <bool PAIR>
bool launch(const CUtensorMap& map_w, const CUtensorMap& map_x, Args a, cudaStream_t s) {
  a.sub_bytes = kXBytes + (a.tile_n / (PAIR ? 2 : 1) * kBlock8 + 1023) / 1024 * 1024;
  a.stage_bytes = kSub * a.sub_bytes;
  a.stages = std::min<int>(kMaxStages, (kSmemMost - 1024 - static_cast<int>(sizeof(Control))) / a.stage_bytes);
  const int smem = 1024 + a.stages * a.stage_bytes + static_cast<int>(sizeof(Control));
  auto kern = k_group_8bit<PAIR>;
  static std::atomic<uint64_t> raised{0};  // devices on which the kernel may use this much shared memory
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(raised.load(std::memory_order_relaxed) & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) != cudaSuccess) return false;
    raised.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sm_count() / 2 * 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {2u, 1u, 1u};
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kern, map_w, map_x, a) == cudaSuccess;
}

// Columns of a tile, and whether two blocks share it (256 rows then, else 128): the least waves x cycles.  A slice takes
// the longer of its instructions (two cycles per column) and its bytes at 60 per cycle and SM; a tile its slices, 1000 to
// change over; a kernel of pairs 2500 to start.  Measured against tiles of 240 columns of a pair, and of 240, 128 and 64 of a
// single block (us; rows as they are, so many groups, matrix):
//    49152 rows, 64, 2048 x 2048   198 against 199, 230, 308, 416      3063 rows, 10,  712 x 992   11.1 against 13.7, 12.3, 13.5, 13.7
//    12288                         75 against 76, 85, 110, 138         1018 rows, 16,  776 x 1024  9.9 against 13.0, 12.0, 10.1, 11.2
//    96                            38 against 48, 39, 51, 59           64 rows, 1,  4096 x 4096    14.6 against 18.5, 21.1, 16.8, 14.7
// (Without the 2500: 15.3 for the 3063 rows and 17.3 for the 64.)  Against all 24 shapes at 14 sizes, in a replayed graph (which
// times short kernels in steps of 2 us): within 1% of the best at 5, within 5% at 6 more; 20% off at 1018 rows of 16 groups (12.3 us,
// 10.3 with 112 to 160 columns), 22% at 20000 rows, 8, 512 x 512 (20.1, 16.4 with 128), 32% at 8 rows, 8, 1024 x 4096 (24.5, 18.5
// with 176 or pairs).
struct Width {
  int n;
  bool pair;
};
thread_local Width t_width = {0, false};  // tests: the width of this thread's calls

Width pick_width(const spgemm_grouping& g, int64_t n, int64_t blocks) {
  if (t_width.n) return t_width;
  const MmaHooks hooks = mma_hooks();
  if (hooks.width) return {std::min(std::max(hooks.width, 32), kMostCols), hooks.pair && hooks.width == 256};
  Width best{kMostCols, true};
  double least = -1.0;
  for (int side = 2; side >= 1; --side)
    for (int cols = kMostCols; cols >= 64; cols -= 16) {
      const int64_t all = mma_likely_tiles(g, 128 * side) * ceil_div(n, cols);
      const double slice = std::max(2.0 * cols, (kXBytes + cols / side * 128.0) / 60.0);
      const double time = std::ceil(static_cast<double>(all) / (sm_count() / side)) * (blocks * slice + 1000.0) + 2500.0 * (side - 1);
      if (least < 0.0 || time < least) {
        least = time;
        best = {cols, side == 2};
      }
    }
  return best;
}

}  // namespace

void mma8_force(int32_t width, int32_t pair) { t_width = {width, pair != 0}; }

bool launch_mma_8bit(const spgemm_grouping& g, const spgemm_rows8& x, const spgemm_weights8& w, const spgemm_dense& y, bool early,
                     cudaStream_t s) {
  if (g.slots == 0) return true;
  const MmaHooks hooks = mma_hooks();
  Args a = {};
  a.offsets = g.offsets;
  a.slots = static_cast<int>(g.slots);
  a.groups = g.groups;
  a.early = early;
  a.n = static_cast<int>(w.rows);
  a.blocks = static_cast<int>(blocks8(w.cols));
  const Width width = pick_width(g, w.rows, a.blocks);
  a.tile_n = width.n;
  a.sx = x.scales;
  a.sx_stride = x.scale_stride;
  a.sw = w.scales;
  a.out = y.data;
  a.out_stride = y.stride;
  a.out_type = y.dtype;
  a.wide = reinterpret_cast<uintptr_t>(y.data) % 16 == 0 && y.stride * dtype_size(y.dtype) % 16 == 0;
  a.err = grouped_err();
  a.polls = hooks.polls > 0 ? static_cast<uint32_t>(hooks.polls) : tc::kMaxPolls;
  a.hold = hooks.hold;
  CUtensorMap map_w, map_x;
  // a single group may carry any group stride: a map wants a multiple of 16 bytes
  const int64_t dims_w[3] = {w.cols, w.rows, w.groups}, dims_x[2] = {x.cols, x.rows};
  const int64_t strides_w[2] = {w.row_stride, w.groups > 1 ? w.group_stride : w.row_stride * w.rows}, strides_x[1] = {x.stride};
  if (!encode_bytes(&map_w, w.values, 3, dims_w, strides_w, static_cast<uint32_t>(width.n / (width.pair ? 2 : 1))) ||
      !encode_bytes(&map_x, x.values, 2, dims_x, strides_x, 128u))
    return false;
  return width.pair ? launch<true>(map_w, map_x, a, s) : launch<false>(map_w, map_x, a, s);
}

}  // namespace sg
