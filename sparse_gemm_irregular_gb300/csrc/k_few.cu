// A whole expert layer for at most 32 tokens, 64 where its matrices are in 8 bits, in four kernels that overlap:
//
//   k_few_logits   logits = x w_router^T
//   k_few_choose   the choice of every token, and the chosen experts with their tokens
//   k_few<up>      h = silu(x G^T) (x U^T)
//   k_few<down>    out[t] = sum_j w_j h_j D^T
//
// The layer reads each chosen expert's matrices once, and is bound by that: a token of 6 experts of 2048 x 1024 reads 75 MB.
// So each warp reads its pieces of the rows straight into registers, in the layout of its matrix instructions, two
// pieces ahead, and asks no other warp until a unit's sums meet.  (Through shared memory, in bulk copies of a row's 256 to 1024
// bytes each, the copies themselves were the bound: 23 cycles each, 3.2 to 3.5 TB/s.)  A block's warps read neighbouring
// pieces: rows of DRAM are read while they are open (each warp with a run of its own: 4.2 TB/s instead of 7.2).  The down
// product's blocks start while the up product's end, and read their first pieces before they wait for the hidden rows.
//
// The hidden rows stay in two 16-bit numbers, what the first leaves in the second, 16 bits of f32's 24 in bf16 and 22 in f16:
// they go through the small matrix instruction, which has room for them, as four tokens' first parts beside their second ones.
// (In one number they cost as much precision as the rounding of the result: 2.4e-3 off in bf16 where 1.7e-3 is the rounding's.)
//
// Products: 16 rows of a matrix times up to 8 tokens, in the small matrix instructions (m16n8k16): the rows of few tokens leave the
// big ones almost empty, and these take their operands from registers.  An expert with more tokens is in the list once
// for every 8 (down: 4), and its matrix comes from L2 again.  (All of an expert's tokens at once, up to 32, want a block per SM for
// their registers: 32 tokens of 64 experts 255 us a layer.)  Up: 8 rows of the gate and the same 8 of up, so that a
// thread has both sums of its hidden values; down: 16 output columns, all experts one after the other.  The contracted index
// is dealt over a block's eight warps in pieces of 256 bytes a row, a lane taking 16 bytes at a time; both operands in the
// same order, so it need not be the memory's.  Matrices in 8 bits are widened in registers, exactly, and multiplied by their block's scale.
// Sums are added in a fixed order: warp by warp, expert by expert.
//
// Measured (a layer in a replayed graph, 2048 x 1024, bf16, top 6 of 64 experts): one token 26 us, 8 tokens 79, 32 tokens 150 (805 MB:
// 5.4 TB/s with the router and the choice); matrices in 8 bits 23, 59 and 109 us: there a piece costs 600 to 700 instructions of its warp,
// half of them to widen it, and what it waits for is not hidden by 16 warps per SM.  A block per SM instead of two: one token 4 us
// more, 8 tokens 26.  The choice takes 6 us and the logits 3, of one token's 26.  One number to a hidden value instead of two: 1 us
// less for one token, 16 for 32.
#include <algorithm>
#include <atomic>

#include "group_mma.h"
#include "quant8.cuh"
#include "route_choice.cuh"

namespace sg {

namespace {

// Against the calls one after the other (2048 x 1024, 10 experts by 3, 64 by 6, 256 by 8; us): 16 bits, 32 tokens 54, 150, 343
// against 63, 153, 340; 64 tokens 73, 178, 466 (one number to a hidden value) against 63, 160, 441.  8 bits, where the calls
// one after the other widen the matrices first: 64 tokens 70, 148, 355 against 103, 376, 1285.
constexpr int kMaxTokens = 64, kMaxTokens16 = 32;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kPerSm = 2;                      // blocks
constexpr int kTile = 8, kHalf = 4;            // rows of x, of h that a piece of a matrix is multiplied with
constexpr int kPieceBytes = 256;               // of a row
constexpr int kLogitTokens = 4;                // of a block of k_few_logits
constexpr int kChooseWarps = 32;               // of k_few_choose

// Up to kTile (or kHalf) tokens of an expert: their hidden rows are first, first + 1, ...
struct alignas(16) Chosen {
  int expert, first, rows, pad;
};

struct ChooseArgs {
  int tokens, experts;
  const float* logits;
  const float* bias;
  spgemm_route_rule rule;
  int32_t* ids;
  float* weights;
  // what the products read: how many pairs of an expert and some of its tokens there are, which (up: kTile of them, down: kHalf),
  // each hidden row's token, and its weight
  int* total;
  Chosen *tiles, *halves;
  int* token;
  float* ordered;
  int* arrived;              // set to 0
  int row_blocks;            // how many of them
};

struct Args {
  int tokens, slots, most;   // most: length of `chosen`
  const int* total;
  const Chosen* chosen;
  const int* token;
  const float* ordered;
  const void* x;             // up: tokens' rows; down: hidden rows, expert by expert
  int64_t x_stride;
  const void* w;
  int64_t w_group, w_row;    // bytes
  const float* scales;       // 8 bits
  int row_blocks, col_blocks;
  int depth, rows;           // contracted length; up: hidden values, down: output columns
  void* out;                 // up: hidden rows, down: out
  int64_t out_stride;
  int sums;                  // bytes in which the warps' sums meet
  int chunks;                // down: blocks that share a unit's pieces
  float* parts;              // down: their sums, [row block][chunk][token][column], where there are several
  int* arrived;              // down: how many are there, by row block
};

template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16<__half>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// two e4m3 numbers in a 16-bit type: exact
template <typename T>
__device__ __forceinline__ uint32_t widen2(uint32_t two);
template <>
__device__ __forceinline__ uint32_t widen2<__half>(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  return static_cast<uint32_t>(h.x) | static_cast<uint32_t>(h.y) << 16;
}
template <>
__device__ __forceinline__ uint32_t widen2<__nv_bfloat16>(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ uint4 load_16(const void* p) { return *static_cast<const uint4*>(p); }
// what is read once: past L1
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

}  // namespace

// A block: one expert, up to four tokens, 32-bit sums; the contracted index is dealt over its threads.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_few_logits(const T* __restrict__ x, int64_t x_stride, const T* __restrict__ w,
                                                         int64_t w_stride, int tokens, int depth, float* __restrict__ logits) {
  __shared__ float s_part[kWarps][kLogitTokens];
  const int e = blockIdx.x, t0 = static_cast<int>(blockIdx.y) * kLogitTokens, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_go();
  float acc[kLogitTokens] = {};
  for (int k = threadIdx.x * 8; k < depth; k += kThreads * 8) {
    const uint4 wv = load_16(w + e * w_stride + k);
    uint4 xv[kLogitTokens];
#pragma unroll
    for (int i = 0; i < kLogitTokens; ++i) xv[i] = load_16(x + min(t0 + i, tokens - 1) * x_stride + k);
#pragma unroll
    for (int i = 0; i < kLogitTokens; ++i)
#pragma unroll
      for (int v = 0; v < 8; ++v)
        acc[i] = fmaf(to_f32(reinterpret_cast<const T*>(&wv)[v]), to_f32(reinterpret_cast<const T*>(&xv[i])[v]), acc[i]);
  }
#pragma unroll
  for (int i = 0; i < kLogitTokens; ++i) {
    const float sum = warp_sum(acc[i]);
    if (lane == 0) s_part[warp][i] = sum;
  }
  __syncthreads();
  if (threadIdx.x < kLogitTokens && t0 + threadIdx.x < tokens) {
    float sum = 0.0f;
#pragma unroll
    for (int o = 0; o < kWarps; ++o) sum += s_part[o][threadIdx.x];
    logits[static_cast<int64_t>(t0 + threadIdx.x) * gridDim.x + e] = sum;
  }
}

// One block: a warp chooses for its token, then the block sorts the choice by experts.
template <int V>
__global__ void __launch_bounds__(kChooseWarps * 32, 1) k_few_choose(const __grid_constant__ ChooseArgs p) {
  extern __shared__ __align__(16) char smem[];
  __shared__ int s_scan[33];
  __shared__ float s_val[kChooseWarps][32];
  const int slots = p.tokens * p.rule.top_k;
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(smem);  // tokens of each expert
  int* first = reinterpret_cast<int*>(mask + p.experts);
  int* ids = first + p.experts;
  float* weights = reinterpret_cast<float*>(ids + slots);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.experts; e += kChooseWarps * 32) mask[e] = 0;
  pdl_wait();
  pdl_go();
  for (int i = threadIdx.x; i < p.row_blocks; i += kChooseWarps * 32) p.arrived[i] = 0;
  for (int t = warp; t < p.tokens; t += kChooseWarps) {
    const int e0 = lane * V;
    float l[V], s[V], bias[V], over;
#pragma unroll
    for (int v = 0; v < V; ++v) bias[v] = p.bias && e0 + v < p.experts ? p.bias[e0 + v] : 0.0f;
    uint32_t chosen;
    load_row<float, 32, V>(p.logits + static_cast<int64_t>(t) * p.experts, p.experts, p.experts % 4 == 0, l);
    const float f = choose<32, V>(p.rule, p.experts / p.rule.groups, l, p.bias != nullptr, bias, s_val[warp], s, &chosen, &over);
    const int mine = __popc(chosen), upto = warp_incl_scan(mine), n = __shfl_sync(0xffffffffu, upto, 31);
    int o = t * p.rule.top_k + upto - mine;
    for (uint32_t left = chosen; left; left &= left - 1, ++o) {
      const int v = __ffs(left) - 1;
      float w = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) w = i == v ? s[i] : w;
      ids[o] = e0 + v;
      weights[o] = w / over * f;
    }
    for (int j = n + lane; j < p.rule.top_k; j += 32) {
      ids[t * p.rule.top_k + j] = -1;
      weights[t * p.rule.top_k + j] = 0.0f;
    }
    __syncwarp();
  }
  __syncthreads();
  for (int i = threadIdx.x; i < slots; i += kChooseWarps * 32) {
    if (ids[i] >= 0) atomicOr(&mask[ids[i]], 1ull << (i / p.rule.top_k));
    p.ids[i] = ids[i];
    p.weights[i] = weights[i];
  }
  __syncthreads();
  // rows of the experts before (up to 64 x 32: 12 bits), how many tiles they make (fewer than 1024 + 2048 / 8: 11 bits) and how many
  // halves more than that (one for every five rows at most: 9 bits)
  const int e = threadIdx.x;
  const unsigned long long m = e < p.experts ? mask[e] : 0ull;
  const int rows = __popcll(m), tiles = (rows + kTile - 1) / kTile, halves = (rows + kHalf - 1) / kHalf;
  const int n = static_cast<int>(rows | static_cast<uint32_t>(tiles) << 12 | static_cast<uint32_t>(halves - tiles) << 23);
  int all = 0;
  const uint32_t before = static_cast<uint32_t>(block_incl_scan(n, s_scan, &all) - n);
  auto tiles_of = [](uint32_t v) { return static_cast<int>(v >> 12 & 0x7ffu); };
  auto halves_of = [&](uint32_t v) { return tiles_of(v) + static_cast<int>(v >> 23); };
  if (m) {
    first[e] = before & 0xfff;
    for (int r = 0; r < rows; r += kTile) p.tiles[tiles_of(before) + r / kTile] = Chosen{e, first[e] + r, min(rows - r, kTile), 0};
    for (int r = 0; r < rows; r += kHalf) p.halves[halves_of(before) + r / kHalf] = Chosen{e, first[e] + r, min(rows - r, kHalf), 0};
  }
  if (threadIdx.x == 0) {
    p.total[0] = tiles_of(all);
    p.total[1] = halves_of(all);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < slots; i += kChooseWarps * 32) {
    if (ids[i] < 0) continue;
    const int t = i / p.rule.top_k, r = first[ids[i]] + __popcll(mask[ids[i]] & ((1ull << t) - 1ull));
    p.ordered[r] = weights[i];
    p.token[r] = t;
  }
}

template <typename T, bool EIGHT, bool DOWN>
__global__ void __launch_bounds__(kThreads, kPerSm) k_few(const __grid_constant__ Args p) {
  extern __shared__ __align__(128) char sums[];
  __shared__ int s_last;                                        // this block is the last of a unit's
  Chosen* list = reinterpret_cast<Chosen*>(sums + p.sums);      // experts ascending
  int* token = reinterpret_cast<int*>(list + p.most);           // of each hidden row
  float* ordered = reinterpret_cast<float*>(token + p.slots);   // its weight
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The choice was complete before the kernel that starts this one early (down) was itself let past its wait; so were the matrices
  // and their scales, which the kernels of this call do not write.
  if (!DOWN) {
    pdl_wait();
    pdl_go();
  }
  // Past L1: every call writes its choice, often at the same addresses, and a line of the one before may have stayed there.
  const int total = __ldcg(p.total);
  for (int i = threadIdx.x; i < p.most; i += kThreads) reinterpret_cast<uint4*>(list)[i] = __ldcg(reinterpret_cast<const uint4*>(p.chosen) + i);
  for (int i = threadIdx.x; i < p.slots; i += kThreads) {
    token[i] = __ldcg(p.token + i);
    if (DOWN) ordered[i] = __ldcg(p.ordered + i);
  }
  if (DOWN)
    for (int i = threadIdx.x; i < p.sums / 4; i += kThreads) reinterpret_cast<float*>(sums)[i] = 0.0f;
  __syncthreads();

  // ---- units: up: 8 hidden values of an expert; down: 16 output columns of all experts, one after the other ---
  constexpr int kSize = EIGHT ? 1 : 2, kDeep = kPieceBytes / kSize;  // numbers of a row's piece
  constexpr int kUnitRows = DOWN ? 16 : 8;
  const int per = (p.rows + kUnitRows - 1) / kUnitRows;      // row blocks of a matrix
  const int pieces = (p.depth + kDeep - 1) / kDeep;          // of a row
  const int step = gridDim.x;
  // Up: a unit is row block b of expert i of the list; down: row block b and chunk i of the pieces of all experts, which are one
  // long row of pieces then.  A block's next unit is `step` units on, a warp takes every eighth piece of one.  No divisions
  // on the way, but down one for a unit's first piece.
  struct Unit {
    int b, i;
  };
  struct Place {
    int i, j, left;  // expert of the list, piece of its rows, pieces to the unit's end (none for this warp: not above 0)
  };
  const int parts = DOWN ? p.chunks : per;  // units with the same expert, or the same row block
  const int step_lo = step % parts, step_hi = step / parts;
  const int span = DOWN ? total * pieces : pieces, share = DOWN ? (span + p.chunks - 1) / p.chunks : pieces;
  auto unit_at = [&](int lo, int hi) { return DOWN ? Unit{hi, lo} : Unit{lo, hi}; };
  auto next_unit = [&](Unit& u) {
    int lo = (DOWN ? u.i : u.b) + step_lo, hi = (DOWN ? u.b : u.i) + step_hi;
    if (lo >= parts) {
      lo -= parts;
      ++hi;
    }
    u = unit_at(lo, hi);
  };
  auto unit_there = [&](const Unit& u) { return DOWN ? u.b < per : u.i < total; };
  auto pieces_of = [&](const Unit& u) { return (DOWN ? min(share, span - u.i * share) : pieces) - warp; };
  auto begin = [&](const Unit& u) {
    if (!DOWN) return Place{u.i, warp, pieces_of(u)};
    const int f = u.i * share + warp;
    return Place{f / pieces, f % pieces, pieces_of(u)};
  };
  auto next_piece = [&](Place& w) {
    w.left -= kWarps;
    w.j += kWarps;
    if (DOWN)
      while (w.j >= pieces) {
        w.j -= pieces;
        ++w.i;
      }
  };
  const Unit first_unit = unit_at(static_cast<int>(blockIdx.x) % parts, static_cast<int>(blockIdx.x) / parts);

  const int g = lane >> 2, q = lane & 3;
  const T* x = static_cast<const T*>(p.x);
  constexpr int kStep = 64 / kSize, kMine = 16 / kSize, kVecs = 16 / (8 * kSize);  // kVecs: 16-byte pieces of x beside 16 bytes of w

  // ---- this warp's pieces, two ahead of their use: four parts of 64 bytes a row, this lane's 16 bytes of each; rows g
  // and g + 8 of the instruction (up: the gate's and up's) ------------------------------------------------------
  // The tokens' rows beside them come along, but for matrices in 8 bits (twice as much of x: no registers for it; half of the
  // next piece's are fetched when a piece is done, the other half while the first is used).
  struct Buffer {
    uint4 lo[4], hi[4];
    uint4 x[EIGHT ? 1 : 4];
    float s_lo[2], s_hi[2];  // 8 bits: scales of two blocks of 128
    int i, j;  // as of a Place; i < 0: nothing here
  };
  int row_b = -1, row_i = -1;
  Unit far_unit = first_unit;
  Place far = begin(far_unit);
  const char *row_lo = nullptr, *row_hi = nullptr;
  auto read_w = [&](Buffer& v) {
    while (far.left <= 0 && unit_there(far_unit)) {  // a chunk may have no piece for this warp
      next_unit(far_unit);
      far = begin(far_unit);
    }
    v.i = unit_there(far_unit) ? far.i : -1;
    v.j = far.j;
    if (v.i < 0) return;
    if (far_unit.b != row_b || far.i != row_i) {
      row_b = far_unit.b;
      row_i = far.i;
      const int r = row_b * kUnitRows + g;  // rows past the end are read as the last one, and not used
      const char* w = static_cast<const char*>(p.w) + list[row_i].expert * p.w_group + q * 16;
      row_lo = w + min(r, p.rows - 1) * p.w_row;
      row_hi = w + (DOWN ? min(r + 8, p.rows - 1) : p.rows + min(r, p.rows - 1)) * p.w_row;
    }
    const int at = far.j * kPieceBytes;
    if (far.j * kDeep + kDeep <= p.depth) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        v.lo[h] = load_once(row_lo + at + h * 64);
        v.hi[h] = load_once(row_hi + at + h * 64);
      }
    } else {  // past the end both operands are zeros
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const bool in = far.j * kDeep + h * kStep + q * kMine < p.depth;
        v.lo[h] = in ? load_once(row_lo + at + h * 64) : make_uint4(0u, 0u, 0u, 0u);
        v.hi[h] = in ? load_once(row_hi + at + h * 64) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
    if constexpr (EIGHT) {
      const float* sc = p.scales + static_cast<int64_t>(list[far.i].expert) * p.row_blocks * p.col_blocks;
      const int r0 = far_unit.b * kUnitRows;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int kb = min(far.j * 2 + h, p.col_blocks - 1);
        v.s_lo[h] = sc[static_cast<int64_t>(r0 / kBlock8) * p.col_blocks + kb];
        v.s_hi[h] = DOWN ? v.s_lo[h] : sc[static_cast<int64_t>((p.rows + r0) / kBlock8) * p.col_blocks + kb];
      }
    }
    next_piece(far);
  };

  // an expert's rows of x for this lane; columns past its tokens hold what nobody looks at
  auto row_of = [&](const Chosen& now) {
    if (DOWN) return x + ((g / kHalf) * p.slots + now.first + min(g % kHalf, now.rows - 1)) * p.x_stride;
    return x + token[now.first + min(g, now.rows - 1)] * p.x_stride;
  };
  constexpr int kEarly = 2;  // 8 bits: parts of the next piece
  uint4 b[EIGHT ? kEarly : 1][kVecs];
  const T* xr = nullptr;
  auto fetch = [&](const Buffer& w, int h) {
    const bool in = w.j * kDeep + kDeep <= p.depth || w.j * kDeep + q * kMine + h * kStep < p.depth;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) b[h % kEarly][v] = in ? load_16(xr + h * kStep + 8 * v) : make_uint4(0u, 0u, 0u, 0u);
  };
  auto read_x = [&](Buffer& v) {
    if (v.i < 0) return;
    const Chosen now = list[v.i];
    const int k = v.j * kDeep + q * kMine;
    if constexpr (EIGHT) {
      xr = row_of(now) + k;
#pragma unroll
      for (int h = 0; h < kEarly; ++h) fetch(v, h);
    } else {
      const bool whole = v.j * kDeep + kDeep <= p.depth;
      const T* from = row_of(now) + k;
#pragma unroll
      for (int h = 0; h < 4; ++h) v.x[h] = whole || k + h * kStep < p.depth ? load_16(from + h * kStep) : make_uint4(0u, 0u, 0u, 0u);
    }
  };

  Unit unit = first_unit;  // the one at hand
  int left = pieces_of(unit);
  int turn = 0;
  int at = -1, first = 0, rows = 0;
  float acc[4] = {};
  // down: this warp's part of the weighted sum: sums[warp][token][column]
  auto add_weighted = [&]() {
    float* mine = reinterpret_cast<float*>(sums) + warp * p.tokens * 16;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = 2 * q + j;
      // h's two parts.  An infinite entry of the matrix times the second one, of either sign or 0, says nothing: the first's is the answer.
      const float rest = __shfl_xor_sync(0xffffffffu, acc[j], 2), rest8 = __shfl_xor_sync(0xffffffffu, acc[2 + j], 2);
      if (fabsf(acc[j]) < INFINITY) acc[j] += rest;
      if (fabsf(acc[2 + j]) < INFINITY) acc[2 + j] += rest8;
      if (r < rows && r < kHalf) {
        float* to = mine + token[first + r] * 16 + g;
        const float w = ordered[first + r];
        to[0] += w * acc[j];
        to[8] += w * acc[2 + j];
      }
      acc[j] = acc[2 + j] = 0.0f;
    }
    __syncwarp();  // a token may be in another row of the next expert, and its sums in another lane's hands
  };
  // the warps' sums of a unit meet
  auto finish = [&]() {
    const int r0 = unit.b * kUnitRows;
    if (DOWN) {
      if (at >= 0) add_weighted();
      __syncthreads();
      float* of = reinterpret_cast<float*>(sums);
      for (int i = threadIdx.x; i < p.tokens * 16; i += kThreads) {
        float sum = 0.0f;
#pragma unroll
        for (int o = 0; o < kWarps; ++o) {
          sum += of[o * p.tokens * 16 + i];
          of[o * p.tokens * 16 + i] = 0.0f;
        }
        if (p.chunks > 1) p.parts[(static_cast<int64_t>(unit.b) * p.chunks + unit.i) * p.tokens * 16 + i] = sum;
        else if (r0 + i % 16 < p.rows) static_cast<T*>(p.out)[(i / 16) * p.out_stride + r0 + i % 16] = from_f32<T>(sum);
      }
      if (p.chunks > 1) {  // the block that comes last adds the chunks up, in their order
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) s_last = atomicAdd(&p.arrived[unit.b], 1) == p.chunks - 1;
        __syncthreads();
        if (s_last) {
          __threadfence();
          for (int i = threadIdx.x; i < p.tokens * 16; i += kThreads) {
            float sum = 0.0f;
            for (int o = 0; o < p.chunks; ++o) sum += __ldcg(&p.parts[(static_cast<int64_t>(unit.b) * p.chunks + o) * p.tokens * 16 + i]);
            if (r0 + i % 16 < p.rows) static_cast<T*>(p.out)[(i / 16) * p.out_stride + r0 + i % 16] = from_f32<T>(sum);
          }
        }
      }
      __syncthreads();
    } else {
      const int first = list[unit.i].first, rows = list[unit.i].rows;
      float4* of = reinterpret_cast<float4*>(sums) + turn * (kWarps * 32);  // [warp][lane]
      of[warp * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
      __syncthreads();
      turn ^= 1;  // the next unit's sums go beside these: one meeting per unit
      if (warp == 0) {
        float4 sum = of[lane];
#pragma unroll
        for (int o = 1; o < kWarps; ++o) {
          const float4 v = of[o * 32 + lane];
          sum.x += v.x;
          sum.y += v.y;
          sum.z += v.z;
          sum.w += v.w;
        }
        T* out = static_cast<T*>(p.out) + (first + 2 * q) * p.out_stride + r0 + g;
        auto put = [&](T* to, float h) {  // what the first part leaves goes into the second
          const T part = from_f32<T>(h);
          const float left = h - to_f32(part);
          to[0] = part;
          to[p.slots * p.out_stride] = from_f32<T>(fabsf(to_f32(part)) < INFINITY ? left : 0.0f);
        };
        if (r0 + g < p.rows) {
          if (2 * q < rows) put(out, gated_silu(sum.x, sum.z));
          if (2 * q + 1 < rows) put(out + p.out_stride, gated_silu(sum.y, sum.w));
        }
      }
    }
    at = -1;
  };
  // one piece, the one behind it in `next`; false: it was the last
  auto work = [&](Buffer& w, Buffer& next) {
    if (DOWN && w.i != at) {
      if (at >= 0) add_weighted();
      at = w.i;
      const Chosen now = list[at];
      first = now.first;
      rows = now.rows;
    }
    float part[4] = {};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const uint4 a = w.lo[h], a8 = w.hi[h];
      if constexpr (!EIGHT) {
        const uint4 v = w.x[h];
        mma16<T>(acc, a.x, a8.x, a.y, a8.y, v.x, v.y);
        mma16<T>(acc, a.z, a8.z, a.w, a8.w, v.z, v.w);
      } else {
        const uint32_t av[4] = {a.x, a.y, a.z, a.w}, av8[4] = {a8.x, a8.y, a8.z, a8.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 v = b[h % kEarly][kVecs - 1 < j / 2 ? 0 : j / 2];
          mma16<T>(part, widen2<T>(av[j] & 0xffffu), widen2<T>(av8[j] & 0xffffu), widen2<T>(av[j] >> 16), widen2<T>(av8[j] >> 16),
                   j % 2 ? v.z : v.x, j % 2 ? v.w : v.y);
        }
        if (h % 2 == 1) {
          acc[0] = fmaf(w.s_lo[h / 2], part[0], acc[0]);
          acc[1] = fmaf(w.s_lo[h / 2], part[1], acc[1]);
          acc[2] = fmaf(w.s_hi[h / 2], part[2], acc[2]);
          acc[3] = fmaf(w.s_hi[h / 2], part[3], acc[3]);
          part[0] = part[1] = part[2] = part[3] = 0.0f;
        }
      }
      if (EIGHT && h + kEarly < 4) fetch(w, h + kEarly);
    }
    read_w(w);
    if (EIGHT) read_x(next);
    else read_x(w);
    left -= kWarps;
    if (left > 0) return true;
    do {  // units without a piece for this warp: it only meets the others
      finish();
      next_unit(unit);
      left = pieces_of(unit);
    } while (left <= 0 && unit_there(unit));
    return unit_there(unit);
  };

  Buffer one, two;
  read_w(one);
  read_w(two);
  if (DOWN) {
    pdl_wait();  // the hidden rows
    pdl_go();
  }
  if (!EIGHT) {
    read_x(one);
    read_x(two);
  }
  while (left <= 0 && unit_there(unit)) {
    finish();
    next_unit(unit);
    left = pieces_of(unit);
  }
  bool more = unit_there(unit);
  if (EIGHT && more) read_x(one);
  while (more) {
    more = work(one, two);
    if (more) more = work(two, one);
  }
}

namespace {

// Length of a list: an expert's last tile may be part of one.
constexpr int64_t most_tiles(int64_t slots, int64_t experts, int tile) { return std::min(slots, std::min(slots, experts) + slots / tile); }

// Shared memory of a block: the warps' sums, the list, each hidden row's token and weight
constexpr int sums_bytes(bool down, int tokens) { return down ? kWarps * tokens * 16 * 4 : 2 * kWarps * 512; }
constexpr int block_bytes(int sums, int most, int slots) { return sums + most * static_cast<int>(sizeof(Chosen)) + 8 * slots; }
constexpr int kMostSlots = kMaxTokens * kMaxTopK;
constexpr int kMostBytes = block_bytes(sums_bytes(true, kMaxTokens), static_cast<int>(most_tiles(kMostSlots, kMaxGroups, kHalf)), kMostSlots);
static_assert(kPerSm * (kMostBytes + 1024) <= 227 * 1024, "blocks of an SM");

template <typename T, bool EIGHT, bool DOWN>
bool launch(Args a, cudaStream_t s) {
  a.sums = sums_bytes(DOWN, a.tokens);
  const int bytes = block_bytes(a.sums, a.most, a.slots);
  auto kern = k_few<T, EIGHT, DOWN>;
  // The limit belongs to the kernel, not to the call: it is raised to the most that any call takes, once per device, and never
  // lowered, so that another thread's call does not take it from under this one's launch.
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(raised.load(std::memory_order_relaxed) & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostBytes) != cudaSuccess) return false;
    raised.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_next(kern, dim3(static_cast<unsigned>(kPerSm * sm_count())), kThreads, static_cast<size_t>(bytes), s, a);
}

// How many blocks share a unit of the down product: the fewest turns of all blocks times pieces of a warp; a unit's end takes
// as long as a piece, with other blocks to meet as three (one token, 6 experts of 1024 x 2048: 29.9 us a layer with one block to a
// unit, 27.6 with two).  The experts that tokens share are not known here.
int down_chunks(int64_t row_blocks, int64_t pieces, int64_t blocks) {
  int best = 1;
  double least = -1.0;
  for (int c = 1; c <= 16; ++c) {
    const double time = ceil_div(row_blocks * c, blocks) * (static_cast<double>(ceil_div(pieces, c * kWarps)) + (c > 1 ? 3.0 : 1.0));
    if (least < 0.0 || time < least) {
      least = time;
      best = c;
    }
  }
  return best;
}

bool matrix_ok(const spgemm_weights* w, const spgemm_weights8* w8) {
  return w ? mma_takes(*w) && w->cols % 8 == 0 : w8->cols % 16 == 0;
}

}  // namespace

bool few_takes(const spgemm_dense& x, const spgemm_dense& w_router, const spgemm_weights* w_up, const spgemm_weights* w_down,
               const spgemm_weights8* up8, const spgemm_weights8* down8) {
  return x.rows <= (up8 ? kMaxTokens : kMaxTokens16) && x.cols % 8 == 0 && mma_takes(x) && mma_takes(w_router) && matrix_ok(w_up, up8) && matrix_ok(w_down, down8);
}

FewScratch few_scratch(const spgemm_dense& x, const spgemm_route_rule& rule, int64_t experts, int64_t hidden, int64_t cols, bool eight) {
  const int64_t slots = x.rows * rule.top_k, most = most_tiles(slots, experts, kHalf), row_blocks = ceil_div(cols, 16);
  const int chunks = down_chunks(row_blocks, most * ceil_div(hidden, kPieceBytes / (eight ? 1 : 2)), static_cast<int64_t>(kPerSm) * sm_count());
  return {4 * x.rows * experts, 4 * slots * hidden, chunks > 1 ? 4 * row_blocks * chunks * x.rows * 16 : 0,
          static_cast<int64_t>(sizeof(Chosen)) * (most_tiles(slots, experts, kTile) + most) + 8 * slots + 8 + 4 * row_blocks, chunks};
}

bool launch_few(const spgemm_dense& x, const spgemm_dense& w_router, const spgemm_route_rule& rule, const float* bias,
                const spgemm_weights* w_up, const spgemm_weights* w_down, const spgemm_weights8* up8, const spgemm_weights8* down8,
                const spgemm_dense& out, int32_t* ids, float* weights, const FewScratch& sizes, float* logits, void* h, float* parts,
                void* lists, cudaStream_t s) {
  const int64_t hidden = w_down ? w_down->cols : down8->cols;
  ChooseArgs r = {};
  r.tokens = static_cast<int>(x.rows);
  r.experts = static_cast<int>(w_router.rows);
  r.logits = logits;
  r.bias = bias;
  r.rule = rule;
  r.ids = ids;
  r.weights = weights;
  Args a = {};
  a.tokens = r.tokens;
  a.slots = r.tokens * rule.top_k;
  const int64_t tiles = most_tiles(a.slots, r.experts, kTile), halves = most_tiles(a.slots, r.experts, kHalf);
  r.tiles = static_cast<Chosen*>(lists);
  r.halves = r.tiles + tiles;
  r.token = reinterpret_cast<int*>(r.halves + halves);
  r.ordered = reinterpret_cast<float*>(r.token + a.slots);
  r.total = reinterpret_cast<int*>(r.ordered + a.slots);
  r.arrived = r.total + 2;
  r.row_blocks = static_cast<int>(ceil_div(out.cols, 16));
  a.token = r.token;
  a.ordered = r.ordered;
  a.chunks = sizes.chunks;
  a.parts = parts;
  a.arrived = r.arrived;
  auto matrix = [&](const spgemm_weights* w, const spgemm_weights8* w8) {
    a.w = w ? w->data : w8->values;
    a.w_group = w ? 2 * w->group_stride : w8->group_stride;
    a.w_row = w ? 2 * w->row_stride : w8->row_stride;
    a.scales = w8 ? w8->scales : nullptr;
    a.row_blocks = w8 ? static_cast<int>(blocks8(w8->rows)) : 0;
    a.col_blocks = w8 ? static_cast<int>(blocks8(w8->cols)) : 0;
  };
  bool ok = true;
  auto go = [&](auto type) {
    using T = decltype(type);
    const dim3 grid(static_cast<unsigned>(r.experts), static_cast<unsigned>(ceil_div(r.tokens, kLogitTokens)));
    const size_t bytes = static_cast<size_t>(12) * r.experts + 8 * static_cast<size_t>(a.slots);
    // 2, 8 or 32 experts a lane (a layer of 64 experts: one token 26.4, 27.3 and 33 us; 64 tokens, 8 bits, 148 us and 154 with 8)
    ok = launch_next(k_few_logits<T>, grid, kThreads, 0, s, static_cast<const T*>(x.data), x.stride, static_cast<const T*>(w_router.data),
                     w_router.stride, r.tokens, static_cast<int>(x.cols), logits) &&
         launch_next(r.experts <= 64 ? k_few_choose<2> : r.experts <= 256 ? k_few_choose<8> : k_few_choose<32>, 1u, kChooseWarps * 32, bytes, s, r);
    a.chosen = r.tiles;
    a.most = static_cast<int>(tiles);
    a.total = r.total;
    matrix(w_up, up8);
    a.x = x.data;
    a.x_stride = x.stride;
    a.depth = static_cast<int>(x.cols);
    a.rows = static_cast<int>(hidden);
    a.out = h;
    a.out_stride = hidden;
    ok = ok && (up8 ? launch<T, true, false>(a, s) : launch<T, false, false>(a, s));
    a.chosen = r.halves;
    a.most = static_cast<int>(halves);
    a.total = r.total + 1;
    matrix(w_down, down8);
    a.x = h;
    a.x_stride = hidden;
    a.depth = static_cast<int>(hidden);
    a.rows = static_cast<int>(out.cols);
    a.out = out.data;
    a.out_stride = out.stride;
    ok = ok && (down8 ? launch<T, true, true>(a, s) : launch<T, false, true>(a, s));
  };
  if (x.dtype == SPGEMM_DTYPE_BF16) go(__nv_bfloat16());
  else go(__half());
  return ok;
}

}  // namespace sg
