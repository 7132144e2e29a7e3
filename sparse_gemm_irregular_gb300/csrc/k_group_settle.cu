// Forward products whose rows leave in 16 bits: the elements that the tensor-core kernel marked are added up again.
//
// y[p, n] is the 32-bit sum of x[row(p), k] w[g][n, k] in the order of k, one fused multiply-add per term, rounded
// once.  The matrix instructions add in another order, so their sum and this one can fall on two sides
// of a rounding boundary, and y (and what is computed from it in 32 bits, the gradient of the weights) would then
// differ by a whole spacing between the two paths: 1.1e-3 of the elements in bf16, 9e-3 in f16 (2048 terms).  So the
// first kernel marks each sum that is no further from a boundary than the two orders may differ, one bit per
// element, and this one computes exactly those in order: 3.5% of a bf16 result, 18% of an f16 one (2048 terms).
//
// A block takes up to 128 rows of one tile and 128 columns (or 64) and passes over the contracted index in 64-deep slices
// through shared memory (only the rows and columns with a mark).  A thread computes an element, up to six at a time,
// from 16-byte pieces of its row and column.  Lane i works i modulo 8 pieces behind: the eight lanes that read together
// are at eight different pieces of 128-byte rows, so they meet different banks whatever their rows and columns
// (all lanes at the same piece, swizzled by row: 5.5 wavefronts per read instead of 3.7).
//
// Bound by shared memory's reads, two of 16 bytes per eight terms, and by the chains of additions: 65536 rows, 2048 x
// 2048, 32 unequal groups: 1.55 ms in bf16, 6.2 ms in f16 (all elements in order on the CUDA cores: 28 ms).
#include <algorithm>
#include <atomic>

#include "group_mma.h"

namespace sg {

namespace {

constexpr int kThreads = 256;
constexpr int kRowsOf = 128;                 // of a block: rows of x
constexpr int kDeep = 64;
constexpr int kEach = 6;                     // elements of a thread at a time
constexpr int kStages = 3;                   // a slice that arrives, the current one, the one before
constexpr int stage_bytes(int cols_of) { return (kRowsOf + cols_of) * kDeep * 2; }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {  // the rest of 16 as zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// acc + x y in one rounding, x and y the lower or upper 16 bits of a word
__device__ __forceinline__ float add_product(float acc, uint32_t x, uint32_t y, __nv_bfloat16) {
  asm("fma.rn.f32.bf16 %0, %1, %2, %0;" : "+f"(acc) : "h"(static_cast<uint16_t>(x)), "h"(static_cast<uint16_t>(y)));
  return acc;
}
__device__ __forceinline__ float add_product(float acc, uint32_t x, uint32_t y, __half) {
  asm("fma.rn.f32.f16 %0, %1, %2, %0;" : "+f"(acc) : "h"(static_cast<uint16_t>(x)), "h"(static_cast<uint16_t>(y)));
  return acc;
}

// acc + the eight products of two 16-byte pieces, in order
template <typename T>
__device__ __forceinline__ float add8(float acc, const uint4& a, const uint4& b) {
  const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = add_product(acc, u[i], v[i], T());
    acc = add_product(acc, u[i] >> 16, v[i] >> 16, T());
  }
  return acc;
}

}  // namespace

template <typename T, int kColsOf>
__global__ void __launch_bounds__(kThreads, 2) k_settle(const int32_t* __restrict__ offsets, int groups, int slots, int tile_n,
                                                     const int32_t* __restrict__ order, int top_k, int64_t x_rows,
                                                     const T* __restrict__ x, int64_t x_stride, const T* __restrict__ w,
                                                     int64_t w_group, int64_t w_row, int depth,
                                                     const uint32_t* __restrict__ unsure, T* __restrict__ y,
                                                     int64_t y_stride, int cols) {
  constexpr int kStage = stage_bytes(kColsOf), kWords = kRowsOf / 32 * kColsOf;
  extern __shared__ __align__(16) unsigned char s_stage[];  // rows of x, then rows of w, per stage
  __shared__ uint32_t s_word[kWords], s_rows[kRowsOf / 32];  // marks: column by column, four words of 32 rows each
  __shared__ int s_pre[kWords], s_tmp[33], s_tile[3];        // marks before each word
  __shared__ const T* s_from[kRowsOf + kColsOf];  // NULL: no mark
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_go();
  // the block's tile: tiles of a group are counted as the first kernel counts them
  const int per = max(tile_n / kRowsOf, 1);  // blocks of a tile
  const int across = (cols + kColsOf - 1) / kColsOf;  // blocks side by side follow one another: they share rows of x and w[g] in L2
  const int tile = static_cast<int>(blockIdx.x) / across / per, sub = static_cast<int>(blockIdx.x) / across % per;
  if (tid == 0) s_tile[0] = -1;
  if (tid < kRowsOf / 32) s_rows[tid] = 0;
  __syncthreads();
  int run = 0;
  for (int g0 = 0; g0 < groups && run <= tile; g0 += kThreads) {
    const int g = g0 + tid;
    int lo = 0, hi = 0;
    if (g < groups) {
      lo = min(max(offsets[g], 0), slots);
      hi = min(max(offsets[g + 1], lo), slots);
    }
    const int n = (hi - lo + tile_n - 1) / tile_n;
    int top = 0;
    const int before = run + block_incl_scan(n, s_tmp, &top) - n;
    if (tile >= before && tile < before + n) {
      const int first = lo + (tile - before) * tile_n + sub * kRowsOf;
      s_tile[0] = g;
      s_tile[1] = first;
      s_tile[2] = min(min(hi - first, tile_n), kRowsOf);
    }
    run += top;
  }
  __syncthreads();
  const int g = s_tile[0], p0 = s_tile[1], rows = s_tile[2];
  if (g < 0 || rows <= 0) return;
  const int m0 = static_cast<int>(blockIdx.x) % across * kColsOf;
  // marks, their counts and the rows and columns that have any
  const int words = (rows + 31) / 32 * kColsOf;
  const int64_t block = static_cast<int64_t>(tile) * ((tile_n + 31) / 32) + sub * (kRowsOf / 32);
  for (int i = tid; i < kWords; i += kThreads) {
    const int j = i / kColsOf, c = i % kColsOf, left = rows - 32 * j;
    uint32_t u = 0;
    if (i < words && m0 + c < cols) u = unsure[(block + j) * cols + m0 + c] & (left >= 32 ? 0xffffffffu : (1u << left) - 1u);
    s_word[c * 4 + j] = u;
    if (u) atomicOr(&s_rows[j], u);
  }
  __syncthreads();
  int total = 0;
  {
    constexpr int kOwn = kWords / kThreads;
    int own = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) own += __popc(s_word[kOwn * tid + i]);
    int before = block_incl_scan(own, s_tmp, &total) - own;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      s_pre[kOwn * tid + i] = before;
      before += __popc(s_word[kOwn * tid + i]);
    }
  }
  if (total == 0) return;
  {
    const T* from = nullptr;
    if (tid < kRowsOf) {
      if ((s_rows[tid / 32] >> (tid % 32)) & 1u) {
        int64_t r = p0 + tid;
        if (order) {
          const int slot = order[r];
          r = slot < 0 ? -1 : slot / top_k;
        }
        if (r >= 0 && r < x_rows) from = x + r * x_stride;
      }
    } else if (tid < kRowsOf + kColsOf) {
      const int c = tid - kRowsOf;
      if (s_word[4 * c] | s_word[4 * c + 1] | s_word[4 * c + 2] | s_word[4 * c + 3])
        from = w + g * w_group + (m0 + c) * w_row;
    }
    if (tid < kRowsOf + kColsOf) s_from[tid] = from;
  }
  __syncthreads();
  const uint32_t stage = static_cast<uint32_t>(__cvta_generic_to_shared(s_stage));
  const int slices = (depth + kDeep - 1) / kDeep;
  // eight threads copy a row's eight pieces: this one always the same piece of the same rows
  constexpr int kCopies = (kRowsOf + kColsOf) * 8 / kThreads;
  const int piece = tid & 7;
  const T* from[kCopies];
#pragma unroll
  for (int i = 0; i < kCopies; ++i) from[i] = s_from[i * (kThreads / 8) + (tid >> 3)];
  const uint32_t to = stage + (tid >> 3) * 128 + (piece << 4);
  auto load = [&](int q) {
    const int k = q * kDeep + piece * 8, left = depth - k;
    if (q < slices && left > 0) {
#pragma unroll
      for (int i = 0; i < kCopies; ++i)
        if (from[i]) copy16(to + q % kStages * kStage + i * (kThreads / 8) * 128, from[i] + k, left >= 8 ? 16u : 2u * left);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int pieces = (depth + 7) / 8, lag = tid & 7;
  for (int b0 = 0; b0 < total; b0 += kThreads * kEach) {
    int xo[kEach], wo[kEach];  // where the element's row and column lie in a stage
    float acc[kEach];
    const int here = min(kEach, (total - b0 - (tid & ~31) + kThreads - 1) / kThreads);  // of this warp
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      acc[e] = 0.0f;
      xo[e] = wo[e] = 0;  // threads without an element read along
      const int i = b0 + e * kThreads + tid;
      if (i < total) {
        int lo = 0, hi = kWords;  // the last word with no more than i marks before it holds mark i
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_pre[mid] <= i) lo = mid;
          else hi = mid;
        }
        uint32_t left = s_word[lo];
        for (int skip = i - s_pre[lo]; skip > 0; --skip) left &= left - 1;
        xo[e] = (lo % 4 * 32 + __ffs(left) - 1) * 128;
        wo[e] = (kRowsOf + lo / 4) * 128;
      }
    }
    load(0);
    for (int q = 0; q <= slices; ++q) {  // the last turn is for the lanes behind
      load(q + 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
      const unsigned char* now = s_stage + q % kStages * kStage;
      const unsigned char* then = s_stage + (q + kStages - 1) % kStages * kStage;
      auto turns = [&](auto checked, auto n) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          if (!checked || static_cast<unsigned>(8 * q + t - lag) < static_cast<unsigned>(pieces)) {
            const unsigned char* at = (t >= lag ? now : then) + (((t - lag) & 7) << 4);
#pragma unroll
            for (int e = 0; e < decltype(n)::value; ++e)
              if (!checked || e < here)
                acc[e] = add8<T>(acc[e], *reinterpret_cast<const uint4*>(at + xo[e]), *reinterpret_cast<const uint4*>(at + wo[e]));
          }
        }
      };
      // a count known to the compiler: reads run ahead of the chains of additions
      if (q == 0 || 8 * q + 8 > pieces) turns(std::true_type(), std::integral_constant<int, kEach>());
      else if (here > 4) turns(std::false_type(), std::integral_constant<int, kEach>());
      else if (here > 3) turns(std::false_type(), std::integral_constant<int, 4>());
      else if (here > 2) turns(std::false_type(), std::integral_constant<int, 3>());
      else if (here > 1) turns(std::false_type(), std::integral_constant<int, 2>());
      else if (here > 0) turns(std::false_type(), std::integral_constant<int, 1>());
      __syncthreads();
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (wo[e]) {
        const int row = xo[e] / 128, col = wo[e] / 128 - kRowsOf;
        if (s_from[row]) y[(p0 + row) * y_stride + m0 + col] = from_f32<T>(acc[e]);
      }
  }
}

bool launch_settle(const spgemm_grouping& g, const spgemm_dense& x, bool gather, const spgemm_weights& w,
                   const spgemm_dense& y, const uint32_t* unsure, int tile_n, cudaStream_t s) {
  if (g.slots == 0 || y.cols == 0) return true;
  bool ok = true;
  const int64_t per = std::max(tile_n / kRowsOf, 1);
  auto go = [&](auto type, auto cols_of) {
    using T = decltype(type);
    constexpr int kColsOf = decltype(cols_of)::value, kSmem = kStages * stage_bytes(kColsOf);
    const int64_t grid = mma_marks_bytes(g, tile_n, 1) / (4 * ceil_div(tile_n, 32)) * per * ceil_div(y.cols, kColsOf);
    if (grid > 0x7fffffff) {
      set_last_error("too many tiles");
      ok = false;
      return;
    }
    static std::atomic<uint64_t> raised{0};  // devices on which the kernel may use this much shared memory
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(raised.load(std::memory_order_relaxed) & bit)) {
      if (cudaFuncSetAttribute(k_settle<T, kColsOf>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) {
        ok = false;
        return;
      }
      raised.fetch_or(bit, std::memory_order_relaxed);
    }
    ok = launch_next(k_settle<T, kColsOf>, static_cast<unsigned>(grid), kThreads, kSmem, s, g.offsets, g.groups,
                     static_cast<int>(g.slots), tile_n, gather ? g.order : nullptr, g.top_k, x.rows,
                     static_cast<const T*>(x.data), x.stride, static_cast<const T*>(w.data), w.group_stride, w.row_stride,
                     static_cast<int>(x.cols), unsure, static_cast<T*>(y.data), y.stride, static_cast<int>(y.cols));
  };
  // Half as wide where that many blocks of 128 columns leave SMs idle: 1018 rows, 16 groups, 1024 x 776 (112 blocks) 75 us
  // with 128 columns, 48 with 64 (f16; bf16 35 and 30); 1018 rows, 1024 x 2048 (256 blocks) 84 and 80 (bf16 43 and 51).
  const bool narrow = mma_likely_tiles(g, tile_n) * per * ceil_div(y.cols, 128) < sm_count();
  for_dtype(x.dtype, [&](auto type) {
    if constexpr (sizeof(type) == 2) {
      if (narrow) go(type, std::integral_constant<int, 64>());
      else go(type, std::integral_constant<int, 128>());
    }
  });
  return ok;
}

}  // namespace sg
