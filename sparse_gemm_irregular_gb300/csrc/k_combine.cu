// Weighted sums of a token's rows in group order, and their gradients.
//
//   out[t] = sum_j w[t,j] y[pos[t,j]]        dy[pos[t,j]] = w[t,j] dout[t]
//   dweights[t,j] = <dout[t], y[pos[t,j]]>
//
// Both are bound by reading (and, for the gradient, writing) the rows once; a row is 16-byte loads by
// consecutive threads when its start and length allow, single elements otherwise.  The sum runs
// over j in order, in 32 bits, so it does not depend on which blocks run when.
#include <algorithm>

#include "groups.h"

namespace sg {

namespace {

constexpr int kThreads = 256;

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T v[V];
};

template <typename T>
bool packs(const spgemm_dense& d, int v) {
  return d.cols % v == 0 && d.stride % v == 0 && reinterpret_cast<uintptr_t>(d.data) % (sizeof(T) * v) == 0;
}

}  // namespace

// One thread per V columns of a token's row.  65536 x 2048 rows to 16384: 90 us from 32-bit rows (604 MB,
// 6.7 TB/s), 65 us from bf16 (335 MB, 5.2 TB/s).
template <typename TY, typename TO, int V>
__global__ void __launch_bounds__(kThreads) k_combine(const int32_t* __restrict__ position, int64_t tokens, int top_k,
                                                      int64_t slots, const float* __restrict__ weights,
                                                      const TY* __restrict__ y, int64_t y_stride, TO* __restrict__ out,
                                                      int64_t out_stride, int64_t cols) {
  pdl_wait();
  pdl_go();
  const int64_t per = cols / V;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < tokens * per;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t t = i / per, c = (i - t * per) * V;
    float acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.0f;
    // 16-bit rows: four at a time, their loads under way before the first is added (65536 x 2048: 65 us against
    // 69); 32-bit rows fill the memory system one at a time (90 us against 99)
    constexpr int kRows = sizeof(TY) == 2 ? 4 : 1;
#pragma unroll 4 / kRows
    for (int j0 = 0; j0 < top_k; j0 += kRows) {
      Pack<TY, V> row[kRows];
      float w[kRows];
      bool there[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const int64_t p = j0 + j < top_k ? position[t * top_k + j0 + j] : -1;
        there[j] = p >= 0 && p < slots;
        w[j] = there[j] && weights ? weights[t * top_k + j0 + j] : 1.0f;
        if (there[j]) row[j] = *reinterpret_cast<const Pack<TY, V>*>(y + p * y_stride + c);
      }
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        if (there[j]) {
#pragma unroll
          for (int v = 0; v < V; ++v) acc[v] += w[j] * to_f32(row[j].v[v]);
        }
    }
    Pack<TO, V> o;
#pragma unroll
    for (int v = 0; v < V; ++v) o.v[v] = from_f32<TO>(acc[v]);
    *reinterpret_cast<Pack<TO, V>*>(out + t * out_stride + c) = o;
  }
}

// One thread per 16 bytes of a token's row: read once, written to each of its positions.  16384 x 2048 rows of
// bf16 to 65536: 48 us, 335 MB at 7.0 TB/s (the writes end in L2).
__global__ void __launch_bounds__(kThreads) k_spread_rows(const int32_t* __restrict__ position, int64_t tokens, int top_k,
                                                          int64_t slots, const uint4* __restrict__ x, int64_t x_stride,
                                                          uint4* __restrict__ out, int64_t out_stride, int per, int rest) {
  pdl_wait();
  pdl_go();
  const int c = blockIdx.y * kThreads + threadIdx.x;
  if (c >= per) return;
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    uint4 v;
    if (rest == 0 || c + 1 < per) {
      v = x[t * x_stride + c];
    } else {  // `rest` elements: the matrix may end with them
      const uint16_t* from = reinterpret_cast<const uint16_t*>(x + t * x_stride + c);
      uint32_t word[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < rest) word[e / 2] |= static_cast<uint32_t>(from[e]) << (e % 2 * 16);
      v = make_uint4(word[0], word[1], word[2], word[3]);
    }
    for (int j = 0; j < top_k; ++j) {
      const int64_t p = position[t * top_k + j];
      if (p >= 0 && p < slots) out[p * out_stride + c] = v;
    }
  }
}

// One block per token: the row of dout is read once per slot, from L1 after the first.  65536 x 2048 in bf16:
// 101 us, 604 MB at 6.0 TB/s.
template <typename T, typename TY, int V>
__global__ void __launch_bounds__(kThreads) k_combine_backward(
    const int32_t* __restrict__ offsets, int groups, const int32_t* __restrict__ position, int64_t tokens, int top_k,
    int64_t slots, const float* __restrict__ weights, const T* __restrict__ dout, int64_t dout_stride,
    const TY* __restrict__ y, int64_t y_stride, T* __restrict__ dy, int64_t dy_stride, float* __restrict__ dweights,
    int64_t cols) {
  __shared__ float s_part[kThreads / 32];
  pdl_wait();
  pdl_go();
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    for (int j = 0; j < top_k; ++j) {
      const int64_t p = position[t * top_k + j];
      float dot = 0.0f;
      if (p >= 0 && p < slots) {
        const float w = weights ? weights[t * top_k + j] : 1.0f;
        for (int64_t c = static_cast<int64_t>(threadIdx.x) * V; c < cols; c += kThreads * V) {
          const Pack<T, V> d = *reinterpret_cast<const Pack<T, V>*>(dout + t * dout_stride + c);
          const Pack<TY, V> r = *reinterpret_cast<const Pack<TY, V>*>(y + p * y_stride + c);
          Pack<T, V> o;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float x = to_f32(d.v[v]);
            dot += x * to_f32(r.v[v]);
            o.v[v] = from_f32<T>(w * x);
          }
          *reinterpret_cast<Pack<T, V>*>(dy + p * dy_stride + c) = o;
        }
      }
      dot = warp_sum(dot);
      if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = dot;
      __syncthreads();
      if (threadIdx.x == 0) {
        float sum = 0.0f;
        for (int w = 0; w < kThreads / 32; ++w) sum += s_part[w];
        dweights[t * top_k + j] = sum;
      }
      __syncthreads();
    }
  }
  // rows behind the last group
  for (int64_t p = max(offsets[groups], 0) + static_cast<int64_t>(blockIdx.x); p < slots; p += gridDim.x)
    for (int64_t c = threadIdx.x; c < cols; c += kThreads) dy[p * dy_stride + c] = from_f32<T>(0.0f);
}

void launch_combine(const spgemm_grouping& g, const float* weights, const spgemm_dense& y, const spgemm_dense& out,
                    cudaStream_t s) {
  const int64_t tokens = out.rows;
  if (tokens == 0 || out.cols == 0) return;
  for_dtype(y.dtype, [&](auto ty) {
    for_dtype(out.dtype, [&](auto to) {
      using TY = decltype(ty);
      using TO = decltype(to);
      auto go = [&](auto v) {
        constexpr int V = decltype(v)::value;
        const int64_t blocks = std::min<int64_t>(ceil_div(tokens * (out.cols / V), kThreads), 1 << 20);
        launch_next(k_combine<TY, TO, V>, static_cast<unsigned>(blocks), kThreads, 0, s, g.position, tokens, g.top_k, g.slots,
                    weights, static_cast<const TY*>(y.data), y.stride, static_cast<TO*>(out.data), out.stride, out.cols);
      };
      constexpr int W = 16 / (sizeof(TY) > sizeof(TO) ? sizeof(TY) : sizeof(TO));
      if (packs<TY>(y, W) && packs<TO>(out, W)) go(std::integral_constant<int, W>());
      else go(std::integral_constant<int, 1>());
    });
  });
}

void launch_spread_rows(const spgemm_grouping& g, const spgemm_dense& x, const spgemm_dense& out, cudaStream_t s) {
  if (g.slots == 0) return;
  const int per = static_cast<int>(ceil_div(x.cols, 8));
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(x.rows, 1 << 20)), static_cast<unsigned>(ceil_div(per, kThreads)));
  launch_next(k_spread_rows, grid, kThreads, 0, s, g.position, x.rows, g.top_k, g.slots, static_cast<const uint4*>(x.data),
              x.stride / 8, static_cast<uint4*>(out.data), out.stride / 8, per, static_cast<int>(x.cols % 8));
}

void launch_combine_backward(const spgemm_grouping& g, const float* weights, const spgemm_dense& dout,
                             const spgemm_dense& y, const spgemm_dense& dy, float* dweights, cudaStream_t s) {
  const int64_t tokens = dout.rows;
  if (tokens == 0) return;
  if (dout.cols == 0) {  // scalar products of no terms
    cudaMemsetAsync(dweights, 0, sizeof(float) * g.slots, s);
    return;
  }
  for_dtype(dout.dtype, [&](auto td) {
    for_dtype(y.dtype, [&](auto ty) {
      using T = decltype(td);
      using TY = decltype(ty);
      auto go = [&](auto v) {
        constexpr int V = decltype(v)::value;
        launch_next(k_combine_backward<T, TY, V>, static_cast<unsigned>(std::min<int64_t>(tokens, 1 << 20)), kThreads, 0, s,
                    g.offsets, g.groups, g.position, tokens, g.top_k, g.slots, weights, static_cast<const T*>(dout.data),
                    dout.stride, static_cast<const TY*>(y.data), y.stride, static_cast<T*>(dy.data), dy.stride, dweights,
                    dout.cols);
      };
      constexpr int W = 16 / (sizeof(TY) > sizeof(T) ? sizeof(TY) : sizeof(T));
      if (packs<T>(dout, W) && packs<TY>(y, W) && packs<T>(dy, W)) go(std::integral_constant<int, W>());
      else go(std::integral_constant<int, 1>());
    });
  });
}

}  // namespace sg
