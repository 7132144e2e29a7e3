// Grouped products on the CUDA cores: any type, stride and alignment.
//
//   forward   y[p, n]  = sum_k x[row(p), k] w[g][n, k]
//   dx        dx[p, k] = sum_n dy[p, n] w[g][n, k]
//   dw        dw[g][n, k] = sum over p of the group of dy[p, n] x[row(p), k]
//
// A 64 x 64 tile of the result per block, 4 x 4 of it per thread, the operands in 16-deep slices
// through shared memory, sums in 32 bits in the order of the contracted index.  Bound by the
// CUDA cores' multiply-adds (and, for few rows, by latency): the path for 32-bit inputs and for rows that
// do not start on 16-byte boundaries, which the copy engine cannot fetch.  65536 rows of 2048 in 32 groups,
// 2048 x 2048: 28 ms a product, 20 TFLOP/s.
#include <algorithm>

#include "groups.h"

namespace sg {

namespace {

constexpr int kTile = 64;
constexpr int kDeep = 16;
constexpr int kThreads = 256;

struct Rows {           // the rows of an operand: x by token, or a matrix by position
  const int32_t* order;  // NULL: row = position
  int top_k;
  int64_t rows;
  __device__ __forceinline__ int64_t row(int64_t p) const {
    if (!order) return p;
    const int32_t s = order[p];
    const int64_t r = s < 0 ? -1 : s / top_k;
    return r < rows ? r : -1;
  }
};

// Offsets as they are used: inside [0, slots] and not decreasing, whatever the array holds.
// No array: one group of all positions.
__device__ __forceinline__ int64_t clamped(const int32_t* offsets, int g, int64_t slots) {
  if (!offsets) return g == 0 ? 0 : slots;
  return min(max(static_cast<int64_t>(offsets[g]), int64_t(0)), slots);
}

// The row tile number `tile` (over all groups, the rest behind the last group counted as group
// `groups`): its group and first and last position.  Every thread gets the answer.
__device__ bool find_tile(const int32_t* __restrict__ offsets, int groups, int64_t slots, int64_t tile, int* group,
                          int64_t* p0, int64_t* p1) {
  __shared__ int64_t s_first[2];
  __shared__ int s_g;
  if (threadIdx.x == 0) {
    int64_t at = 0, lo = 0;
    s_g = -1;
    for (int g = 0; g <= groups; ++g) {
      lo = max(lo, clamped(offsets, g, slots));
      const int64_t hi = g < groups ? max(lo, clamped(offsets, g + 1, slots)) : slots;
      const int64_t n = ceil_div(hi - lo, kTile);
      if (tile < at + n) {
        s_g = g;
        s_first[0] = lo + (tile - at) * kTile;
        s_first[1] = min(hi, s_first[0] + kTile);
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  *group = s_g;
  *p0 = s_first[0];
  *p1 = s_first[1];
  return s_g >= 0;
}

// acc[4][4] += a(m, k) * b(n, k) over k in [0, depth) for the thread's rows m and n of the tile.
template <typename FA, typename FB>
__device__ __forceinline__ void tile_product(int64_t depth, FA a, FB b, float (&acc)[4][4]) {
  __shared__ float s_a[kDeep][kTile + 1], s_b[kDeep][kTile + 1];
  const int tm = (threadIdx.x / 16) * 4, tn = (threadIdx.x % 16) * 4;
  for (int64_t k0 = 0; k0 < depth; k0 += kDeep) {
    for (int i = threadIdx.x; i < kTile * kDeep; i += kThreads) {
      a.fill(s_a, i, k0, depth);
      b.fill(s_b, i, k0, depth);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      float x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = s_a[k][tm + i];
        y[i] = s_b[k][tn + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += x[i] * y[j];
    }
    __syncthreads();
  }
}

// Slice loaders.  ByRow: element (m, k) at base[row(m) * stride + k]; ByCol: base[row(k) * stride + m].
template <typename T>
struct ByRow {
  const T* base;
  int64_t stride, first, end;  // rows [first, end) of the tile
  Rows rows;
  __device__ __forceinline__ void fill(float (&s)[kDeep][kTile + 1], int i, int64_t k0, int64_t depth) const {
    const int k = i % kDeep, m = i / kDeep;
    const int64_t p = first + m;
    const int64_t r = p < end ? rows.row(p) : -1;
    s[k][m] = r >= 0 && k0 + k < depth ? to_f32(base[r * stride + k0 + k]) : 0.0f;
  }
};
template <typename T>
struct ByCol {
  const T* base;
  int64_t stride, first, end;  // columns [first, end) of the tile
  int64_t start;               // position of contracted index 0
  Rows rows;
  __device__ __forceinline__ void fill(float (&s)[kDeep][kTile + 1], int i, int64_t k0, int64_t depth) const {
    const int m = i % kTile, k = i / kTile;
    const int64_t r = k0 + k < depth ? rows.row(start + k0 + k) : -1;
    s[k][m] = r >= 0 && first + m < end ? to_f32(base[r * stride + first + m]) : 0.0f;
  }
};

}  // namespace

// forward (BT = false: w rows are the output columns) and dx (BT = true: w columns are)
template <typename T, typename TO, bool BT>
__global__ void __launch_bounds__(kThreads) k_plain_rows(const int32_t* __restrict__ offsets, int groups, int64_t slots,
                                                         Rows rows, const T* __restrict__ x, int64_t x_stride,
                                                         const T* __restrict__ w, int64_t w_group, int64_t w_row,
                                                         int64_t depth, TO* __restrict__ y, int64_t y_stride,
                                                         int64_t cols) {
  int g;
  int64_t p0, p1;
  if (!find_tile(offsets, groups, slots, blockIdx.x, &g, &p0, &p1)) return;
  const int64_t n0 = static_cast<int64_t>(blockIdx.y) * kTile;
  float acc[4][4] = {};
  if (g < groups) {
    const T* wg = w + g * w_group;
    const ByRow<T> a{x, x_stride, p0, p1, rows};
    if (BT) tile_product(depth, a, ByCol<T>{wg, w_row, n0, cols, 0, Rows{nullptr, 1, 0}}, acc);
    else tile_product(depth, a, ByRow<T>{wg, w_row, n0, cols, Rows{nullptr, 1, 0}}, acc);
  }
  const int tm = (threadIdx.x / 16) * 4, tn = (threadIdx.x % 16) * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (p0 + tm + i < p1 && n0 + tn + j < cols) y[(p0 + tm + i) * y_stride + n0 + tn + j] = from_f32<TO>(acc[i][j]);
}

// dw: one group per grid.z, contracted over its positions
template <typename T>
__global__ void __launch_bounds__(kThreads) k_plain_dw(const int32_t* __restrict__ offsets, int groups, int64_t slots,
                                                       Rows rows, const T* __restrict__ dy, int64_t dy_stride,
                                                       const T* __restrict__ x, int64_t x_stride, T* __restrict__ dw,
                                                       int64_t dw_group, int64_t dw_row, int64_t n, int64_t k) {
  const int g = blockIdx.z;
  const int64_t p0 = clamped(offsets, g, slots), p1 = max(p0, clamped(offsets, g + 1, slots));
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kTile, k0 = static_cast<int64_t>(blockIdx.y) * kTile;
  float acc[4][4] = {};
  tile_product(p1 - p0, ByCol<T>{dy, dy_stride, n0, n, p0, Rows{nullptr, 1, 0}}, ByCol<T>{x, x_stride, k0, k, p0, rows},
               acc);
  const int tm = (threadIdx.x / 16) * 4, tn = (threadIdx.x % 16) * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n0 + tm + i < n && k0 + tn + j < k)
        dw[g * dw_group + (n0 + tm + i) * dw_row + k0 + tn + j] = from_f32<T>(acc[i][j]);
}

// silu(gate) * up of 32-bit sums; one element per thread, bound by memory.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_gated(const float* __restrict__ pre, int64_t rows, int64_t hidden,
                                                    T* __restrict__ h, int64_t h_stride) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < rows * hidden;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t r = i / hidden, c = i - r * hidden;
    const float* p = pre + r * 2 * hidden + c;
    h[r * h_stride + c] = from_f32<T>(gated_silu(p[0], p[hidden]));
  }
}

// The adapter's second product, one element per thread over the rank: bound by the CUDA cores.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_adapter_add(const int32_t* __restrict__ position, int64_t slots,
                                                          const int32_t* __restrict__ ids, int groups,
                                                          const float* __restrict__ scale,
                                                          const float* __restrict__ base, const float* __restrict__ v,
                                                          int64_t rank, const T* __restrict__ b, int64_t b_group,
                                                          int64_t b_row, T* __restrict__ y, int64_t y_stride,
                                                          int64_t cols) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < slots * cols;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t t = i / cols, n = i - t * cols;
    float sum = 0.0f;
    const int64_t p = position[t];
    if (p >= 0 && p < slots) {
      const int g = ids[t];
      const T* row = b + g * b_group + n * b_row;
      for (int64_t r = 0; r < rank; ++r) sum += v[p * rank + r] * to_f32(row[r]);
      if (scale) sum *= scale[g];
    }
    y[t * y_stride + n] = from_f32<T>(base[i] + sum);
  }
}

namespace {

unsigned row_tiles(const spgemm_grouping& g) {
  return static_cast<unsigned>(ceil_div(g.slots, kTile) + g.groups + 1);  // each group ends in a part tile
}

unsigned flat_blocks(int64_t n) { return static_cast<unsigned>(std::min<int64_t>(ceil_div(n, kThreads), 1 << 20)); }

}  // namespace

void launch_plain_forward(const spgemm_grouping& g, const spgemm_dense& x, bool gather, const spgemm_weights& w,
                          const spgemm_dense& y, cudaStream_t s) {
  if (g.slots == 0 || y.cols == 0) return;
  const dim3 grid(row_tiles(g), static_cast<unsigned>(ceil_div(y.cols, kTile)));
  const Rows rows{gather ? g.order : nullptr, g.top_k, x.rows};
  for_dtype(x.dtype, [&](auto tx) {
    using T = decltype(tx);
    auto go = [&](auto to) {
      using TO = decltype(to);
      note_launch();
      k_plain_rows<T, TO, false><<<grid, kThreads, 0, s>>>(
          g.offsets, g.groups, g.slots, rows, static_cast<const T*>(x.data), x.stride, static_cast<const T*>(w.data),
          w.group_stride, w.row_stride, w.cols, static_cast<TO*>(y.data), y.stride, y.cols);
    };
    if (y.dtype == SPGEMM_DTYPE_F32) go(float());
    else go(T());
  });
}

void launch_plain_dx(const spgemm_grouping& g, const spgemm_dense& dy, const spgemm_weights& w, float* dx,
                     cudaStream_t s) {
  if (g.slots == 0 || w.cols == 0) return;
  const dim3 grid(row_tiles(g), static_cast<unsigned>(ceil_div(w.cols, kTile)));
  for_dtype(dy.dtype, [&](auto t) {
    using T = decltype(t);
    note_launch();
    k_plain_rows<T, float, true><<<grid, kThreads, 0, s>>>(
        g.offsets, g.groups, g.slots, Rows{nullptr, 1, dy.rows}, static_cast<const T*>(dy.data), dy.stride,
        static_cast<const T*>(w.data), w.group_stride, w.row_stride, w.rows, dx, w.cols, w.cols);
  });
}

void launch_plain_dw(const spgemm_grouping& g, const spgemm_dense& dy, const spgemm_dense& x, const spgemm_weights& dw,
                     cudaStream_t s) {
  if (dw.rows == 0 || dw.cols == 0) return;
  const dim3 grid(static_cast<unsigned>(ceil_div(dw.rows, kTile)), static_cast<unsigned>(ceil_div(dw.cols, kTile)),
                  static_cast<unsigned>(g.groups));
  for_dtype(x.dtype, [&](auto t) {
    using T = decltype(t);
    note_launch();
    k_plain_dw<T><<<grid, kThreads, 0, s>>>(g.offsets, g.groups, g.slots, Rows{g.order, g.top_k, x.rows},
                                            static_cast<const T*>(dy.data), dy.stride, static_cast<const T*>(x.data),
                                            x.stride, static_cast<T*>(dw.data), dw.group_stride, dw.row_stride, dw.rows,
                                            dw.cols);
  });
}

void launch_gated(const float* pre, int64_t rows, int64_t hidden, const spgemm_dense& h, cudaStream_t s) {
  if (rows * hidden == 0) return;
  for_dtype(h.dtype, [&](auto t) {
    using T = decltype(t);
    note_launch();
    k_gated<T><<<flat_blocks(rows * hidden), kThreads, 0, s>>>(pre, rows, hidden, static_cast<T*>(h.data), h.stride);
  });
}

void launch_plain_adapter_add(const spgemm_grouping& g, const int32_t* ids, const float* scale, const float* base,
                              const float* v, int64_t rank, const spgemm_weights& b, const spgemm_dense& y,
                              cudaStream_t s) {
  if (y.rows * y.cols == 0) return;
  for_dtype(y.dtype, [&](auto t) {
    using T = decltype(t);
    note_launch();
    k_adapter_add<T><<<flat_blocks(y.rows * y.cols), kThreads, 0, s>>>(
        g.position, g.slots, ids, g.groups, scale, base, v, rank, static_cast<const T*>(b.data), b.group_stride,
        b.row_stride, static_cast<T*>(y.data), y.stride, y.cols);
  });
}

}  // namespace sg
