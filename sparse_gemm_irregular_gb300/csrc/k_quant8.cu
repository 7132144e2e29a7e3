// Rows and matrices in 8-bit floating point with a scale per block (quant8.cuh): made, read back, laid out in group order;
// and the gated product of a training step, whose backward pass reads gate and up from their 8 bits.
//
//   h = silu(g) u                      (forward, from the numbers themselves)
//   dg = dh u s (1 + g (1 - s)),  du = dh g s,  h = g s u with s = 1 / (1 + exp(-g))     (backward, from 8 bits)
//
// All of them read and write each number once and are bound by that.  16 lanes hold a block, eight numbers (16 bytes of
// a 16-bit type) each, so that a block's largest magnitude is four shuffles away and nothing waits for another warp.
#include <algorithm>
#include <type_traits>

#include "group_mma.h"
#include "quant8.cuh"

namespace sg {

namespace {

constexpr int kThreads = 256;
constexpr int kRowsOf = kThreads / 32;   // rows of a block: one a warp, two blocks of a row at a time
constexpr int64_t kBlocksPerSm = 16;     // of the grid, where there are rows for several a warp

// f(p) for every position p of token t, read by the lanes at once; the whole warp calls it.
template <typename F>
__device__ __forceinline__ void at_positions(const int32_t* __restrict__ position, int64_t t, int top_k, int64_t slots, F f) {
  const int lane = threadIdx.x & 31, mine = lane < top_k ? position[t * top_k + lane] : -1;
  for (int j = 0; j < top_k; ++j) {
    const int p = __shfl_sync(0xffffffffu, mine, j);
    if (p >= 0 && p < slots) f(p);
  }
}

}  // namespace

// q = x in 8 bits; with `position` (top_k > 0) each row goes to all positions of its token, else to its own place.  65536 x 2048
// bf16: 86 us, 403 MB at 4.7 TB/s; 32768 x 2048 f32 55 us, 336 MB at 6.1 TB/s.  (Back in bf16: 82 us.)
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_quantise_rows(const T* __restrict__ x, int64_t x_stride, bool whole, int64_t rows, int64_t cols,
                    const int32_t* __restrict__ position, int top_k, int64_t slots, uint8_t* __restrict__ q, int64_t q_stride,
                    float* __restrict__ scales, int64_t scale_stride) {
  pdl_wait();
  pdl_go();
  const int lane = threadIdx.x & 31;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * kPiece, b = c / kBlock8;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRowsOf + (threadIdx.x >> 5); t < rows;
       t += static_cast<int64_t>(gridDim.x) * kRowsOf) {
    float v[kPiece];
    load_piece(x + t * x_stride, c, cols, whole, v);
    Scale8 s;
    const uint2 w = quantise_block(v, most_of_block(most_of(v)), &s);
    auto put = [&](int64_t p) {
      if (c >= cols) return;
      store_piece8(q + p * q_stride, c, cols, w);
      if (lane % 16 == 0) scales[b * scale_stride + p] = s.scale;
    };
    if (position) at_positions(position, t, top_k, slots, put);
    else put(t);
  }
}

// Rows that are in 8 bits already, to all positions of their tokens.
__global__ void __launch_bounds__(kThreads)
    k_lay_rows8(const uint8_t* __restrict__ x, int64_t x_stride, const float* __restrict__ x_scales, int64_t x_scale_stride,
                int64_t tokens, int64_t cols, const int32_t* __restrict__ position, int top_k, int64_t slots,
                uint8_t* __restrict__ q, int64_t q_stride, float* __restrict__ scales, int64_t scale_stride) {
  pdl_wait();
  pdl_go();
  const int lane = threadIdx.x & 31;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * kPiece, b = c / kBlock8;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRowsOf + (threadIdx.x >> 5); t < tokens;
       t += static_cast<int64_t>(gridDim.x) * kRowsOf) {
    const uint2 w = c < cols ? load_piece8(x + t * x_stride, c, cols) : make_uint2(0u, 0u);
    const float s = c < cols ? x_scales[b * x_scale_stride + t] : 0.0f;
    at_positions(position, t, top_k, slots, [&](int64_t p) {
      if (c >= cols) return;
      store_piece8(q + p * q_stride, c, cols, w);
      if (lane % 16 == 0) scales[b * scale_stride + p] = s;
    });
  }
}

// out = what the 8 bits stand for; with `position` each row goes to all positions of its token.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_dequantise_rows(const uint8_t* __restrict__ q, int64_t q_stride, const float* __restrict__ scales, int64_t scale_stride,
                      int64_t rows, int64_t cols, const int32_t* __restrict__ position, int top_k, int64_t slots,
                      T* __restrict__ out, int64_t out_stride, bool whole) {
  pdl_wait();
  pdl_go();
  const int lane = threadIdx.x & 31;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * kPiece, b = c / kBlock8;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRowsOf + (threadIdx.x >> 5); t < rows;
       t += static_cast<int64_t>(gridDim.x) * kRowsOf) {
    float v[kPiece] = {};
    if (c < cols) dequantise_piece(load_piece8(q + t * q_stride, c, cols), scales[b * scale_stride + t], v);
#pragma unroll
    for (int e = 0; e < kPiece; ++e) v[e] = held<T>(v[e]);
    auto put = [&](int64_t p) {
      if (c < cols) store_piece(out + p * out_stride, c, cols, whole, v);
    };
    if (position) at_positions(position, t, top_k, slots, put);
    else put(t);
  }
}

// A block of threads makes one block of 128 x 128: 16 rows at a time, the numbers stay in registers until the largest
// of them all is known.  64 matrices of 2048 x 2048, bf16: 698 us, 805 MB at 1.2 TB/s, the copy rate 119 us; 16 of them in 32 bits
// 112 us, 336 MB at 3.0 TB/s.  Its registers (140) leave an SM one such block, which reads, meets and writes by turns; it runs once, when a
// program lays its weights out.  (Back in bf16, below: 144 us, 5.6 TB/s.)
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_quantise_weights(const T* __restrict__ w, int64_t group_stride, int64_t row_stride, bool whole, int64_t rows, int64_t cols,
                       int64_t row_blocks, int64_t col_blocks, uint8_t* __restrict__ q, int64_t q_group, int64_t q_stride,
                       float* __restrict__ scales) {
  constexpr int kTurns = kBlock8 / (kThreads / 16);
  __shared__ uint32_t s_most[kThreads / 32];
  pdl_wait();
  pdl_go();
  const int64_t at = blockIdx.x, cb = at % col_blocks, rb = at / col_blocks % row_blocks, g = at / col_blocks / row_blocks;
  const int64_t c = cb * kBlock8 + (threadIdx.x % 16) * kPiece, r0 = rb * kBlock8 + threadIdx.x / 16;
  float v[kTurns][kPiece];
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int64_t r = r0 + i * (kThreads / 16);
    if (r < rows) {
      load_piece(w + g * group_stride + r * row_stride, c, cols, whole, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < kPiece; ++e) v[i][e] = 0.0f;
    }
    most = max(most, most_of(v[i]));
  }
  auto of_all = [&](uint32_t m) {
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) s_most[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = max(m, s_most[i]);
    __syncthreads();
    return m;
  };
  most = of_all(most);
  if (!all_finite(most)) {  // all threads alike
    most = 0;
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      most = max(most, most_finite_of(v[i]));
#pragma unroll
      for (int e = 0; e < kPiece; ++e) v[i][e] = fabsf(v[i][e]) < INFINITY ? v[i][e] : NAN;
    }
    most = of_all(most);
  }
  const Scale8 s = scale_of(most);
  if (threadIdx.x == 0) scales[at] = s.scale;
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int64_t r = r0 + i * (kThreads / 16);
    if (r < rows) store_piece8(q + g * q_group + r * q_stride, c, cols, quantise_piece(v[i], s.inverse));
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_dequantise_weights(const uint8_t* __restrict__ q, int64_t q_group, int64_t q_stride, const float* __restrict__ scales,
                         int64_t rows, int64_t cols, int64_t row_blocks, int64_t col_blocks, T* __restrict__ w,
                         int64_t group_stride, int64_t row_stride, bool whole) {
  constexpr int kTurns = kBlock8 / (kThreads / 16);
  pdl_wait();
  pdl_go();
  const int64_t at = blockIdx.x, cb = at % col_blocks, rb = at / col_blocks % row_blocks, g = at / col_blocks / row_blocks;
  const int64_t c = cb * kBlock8 + (threadIdx.x % 16) * kPiece, r0 = rb * kBlock8 + threadIdx.x / 16;
  const float s = scales[at];
  if (c >= cols) return;
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int64_t r = r0 + i * (kThreads / 16);
    if (r >= rows) break;
    float v[kPiece];
    dequantise_piece(load_piece8(q + g * q_group + r * q_stride, c, cols), s, v);
#pragma unroll
    for (int e = 0; e < kPiece; ++e) v[e] = held<T>(v[e]);
    store_piece(w + g * group_stride + r * row_stride, c, cols, whole, v);
  }
}

// 65536 rows, 1024 hidden, bf16: 102 us, 537 MB at 5.3 TB/s (142 us while a warp had one row and looked at each magnitude for
// infinity, with exponentials and divisions of 32 bits); rows in 32 bits and h in bf16 123 us, 805 MB at 6.5 TB/s
template <typename T, typename TO>
__global__ void __launch_bounds__(kThreads)
    k_gated8(const T* __restrict__ pre, int64_t pre_stride, bool whole_gate, bool whole_up, int64_t rows, int64_t hidden,
             TO* __restrict__ h, int64_t h_stride, bool whole_h, uint8_t* __restrict__ gate, int64_t gate_stride,
             float* __restrict__ gate_scales, int64_t gate_scale_stride, uint8_t* __restrict__ up, int64_t up_stride,
             float* __restrict__ up_scales, int64_t up_scale_stride) {
  pdl_wait();
  pdl_go();
  const int lane = threadIdx.x & 31;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * kPiece, b = c / kBlock8;
  int64_t r = static_cast<int64_t>(blockIdx.x) * kRowsOf + (threadIdx.x >> 5);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRowsOf;
  // addresses move along with the row
  pre += r * pre_stride;
  h += r * h_stride;
  gate += r * gate_stride;
  up += r * up_stride;
  gate_scales += b * gate_scale_stride + r;
  up_scales += b * up_scale_stride + r;
  for (; r < rows; r += step) {
    float g[kPiece], u[kPiece], o[kPiece];
    load_piece(pre, c, hidden, whole_gate, g);
    load_piece(pre + hidden, c, hidden, whole_up, u);
    Scale8 sg, su;
    const uint32_t most_gate = most_of_block(most_of(g));
    const uint2 g8 = quantise_block(g, most_gate, &sg), u8 = quantise_block(u, most_of_block(most_of(u)), &su);
    if (c < hidden) {
      auto product = [&](auto is_short) {
#pragma unroll
        for (int e = 0; e < kPiece; ++e) o[e] = g[e] * sigmoid<decltype(is_short)::value>(g[e]) * u[e];
      };
      // (magnitudes compare as their bits do; what is not finite is above all)
      if (sizeof(TO) == 2 && most_gate <= __float_as_uint(kShortGate)) product(std::true_type());
      else product(std::false_type());
      store_piece(h, c, hidden, whole_h, o);
      store_piece8(gate, c, hidden, g8);
      store_piece8(up, c, hidden, u8);
      if (lane % 16 == 0) {
        *gate_scales = sg.scale;
        *up_scales = su.scale;
      }
    }
    pre += step * pre_stride;
    h += step * h_stride;
    gate += step * gate_stride;
    up += step * up_stride;
    gate_scales += step;
    up_scales += step;
  }
}

// 65536 rows, 1024 hidden, bf16: 112 us, 671 MB at 6.0 TB/s
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_gated8_backward(const T* __restrict__ dh, int64_t dh_stride, bool whole_dh, int64_t rows, int64_t hidden,
                      const uint8_t* __restrict__ gate, int64_t gate_stride, const float* __restrict__ gate_scales,
                      int64_t gate_scale_stride, const uint8_t* __restrict__ up, int64_t up_stride,
                      const float* __restrict__ up_scales, int64_t up_scale_stride, T* __restrict__ dpre, int64_t dpre_stride,
                      bool whole_gate, bool whole_up, T* __restrict__ h, int64_t h_stride, bool whole_h) {
  pdl_wait();
  pdl_go();
  const int lane = threadIdx.x & 31;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * kPiece, b = c / kBlock8;
  if (c >= hidden) return;
  int64_t r = static_cast<int64_t>(blockIdx.x) * kRowsOf + (threadIdx.x >> 5);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRowsOf;
  const bool again = h != nullptr;
  dh += r * dh_stride;
  gate += r * gate_stride;
  up += r * up_stride;
  gate_scales += b * gate_scale_stride + r;
  up_scales += b * up_scale_stride + r;
  dpre += r * dpre_stride;
  h += r * h_stride;
  for (; r < rows; r += step) {
    float g[kPiece], u[kPiece], d[kPiece], dg[kPiece], du[kPiece], o[kPiece];
    load_piece(dh, c, hidden, whole_dh, d);
    const float gate_scale = *gate_scales;
    dequantise_piece(load_piece8(gate, c, hidden), gate_scale, g);
    dequantise_piece(load_piece8(up, c, hidden), *up_scales, u);
    auto product = [&](auto is_short) {
#pragma unroll
      for (int e = 0; e < kPiece; ++e) {
        const float s = sigmoid<decltype(is_short)::value>(g[e]), gs = g[e] * s;
        o[e] = gs * u[e];
        du[e] = d[e] * gs;
        dg[e] = d[e] * u[e] * (s + gs * (1.0f - s));
      }
    };
    // no number of the block is above 448 of its scale
    if (sizeof(T) == 2 && fabsf(gate_scale) <= kShortGate / 448.0f) product(std::true_type());
    else product(std::false_type());
    store_piece(dpre, c, hidden, whole_gate, dg);
    store_piece(dpre + hidden, c, hidden, whole_up, du);
    if (again) store_piece(h, c, hidden, whole_h, o);
    dh += step * dh_stride;
    gate += step * gate_stride;
    up += step * up_stride;
    gate_scales += step;
    up_scales += step;
    dpre += step * dpre_stride;
    h += step * h_stride;
  }
}

namespace {

bool on_16(const void* data, int64_t stride, int32_t dtype, int64_t offset = 0) {
  const int64_t size = dtype_size(dtype);
  return reinterpret_cast<uintptr_t>(data) % 16 == 0 && stride * size % 16 == 0 && offset * size % 16 == 0;
}

// A warp per row and 256 columns; with enough of them, several rows a warp.  Forward and backward of 65536 rows, 1024 hidden: 16
// blocks per SM 102 and 112 us, 8 of them 103 and 111, 64 of them 107 and 117, a warp for every row 119 and 129.
dim3 row_grid(int64_t rows, int64_t cols) {
  const int64_t across = ceil_div(cols, 2 * kBlock8), down = ceil_div(rows, kRowsOf);
  return dim3(static_cast<unsigned>(std::min(down, std::max<int64_t>(1, kBlocksPerSm * sm_count() / across))), static_cast<unsigned>(across));
}

uint8_t* bytes(void* p) { return static_cast<uint8_t*>(p); }

}  // namespace

void launch_quantise_rows(const spgemm_dense& x, const spgemm_grouping* g, const spgemm_rows8& q, cudaStream_t s) {
  if (x.rows == 0 || x.cols == 0) return;
  for_dtype(x.dtype, [&](auto type) {
    using T = decltype(type);
    launch_next(k_quantise_rows<T>, row_grid(x.rows, x.cols), kThreads, 0, s, static_cast<const T*>(x.data), x.stride,
                on_16(x.data, x.stride, x.dtype), x.rows, x.cols, g ? g->position : nullptr, g ? g->top_k : 0,
                g ? g->slots : 0, bytes(q.values), q.stride, q.scales, q.scale_stride);
  });
}

void launch_lay_rows8(const spgemm_rows8& x, const spgemm_grouping& g, const spgemm_rows8& q, cudaStream_t s) {
  if (x.rows == 0 || x.cols == 0) return;
  launch_next(k_lay_rows8, row_grid(x.rows, x.cols), kThreads, 0, s, bytes(x.values), x.stride, x.scales, x.scale_stride, x.rows,
              x.cols, g.position, g.top_k, g.slots, bytes(q.values), q.stride, q.scales, q.scale_stride);
}

void launch_dequantise_rows(const spgemm_rows8& q, const spgemm_grouping* g, const spgemm_dense& out, cudaStream_t s) {
  if (q.rows == 0 || q.cols == 0) return;
  for_dtype(out.dtype, [&](auto type) {
    using T = decltype(type);
    launch_next(k_dequantise_rows<T>, row_grid(q.rows, q.cols), kThreads, 0, s, bytes(q.values), q.stride, q.scales,
                q.scale_stride, q.rows, q.cols, g ? g->position : nullptr, g ? g->top_k : 0, g ? g->slots : 0,
                static_cast<T*>(out.data), out.stride, on_16(out.data, out.stride, out.dtype));
  });
}

void launch_quantise_weights(const spgemm_weights& w, const spgemm_weights8& q, cudaStream_t s) {
  const int64_t rb = blocks8(w.rows), cb = blocks8(w.cols);
  for_dtype(w.dtype, [&](auto type) {
    using T = decltype(type);
    const bool whole = on_16(w.data, w.row_stride, w.dtype, w.group_stride);
    launch_next(k_quantise_weights<T>, dim3(static_cast<unsigned>(w.groups * rb * cb)), kThreads, 0, s,
                static_cast<const T*>(w.data), w.group_stride, w.row_stride, whole, w.rows, w.cols, rb, cb, bytes(q.values),
                q.group_stride, q.row_stride, q.scales);
  });
}

void launch_dequantise_weights(const spgemm_weights8& q, const spgemm_weights& w, cudaStream_t s) {
  const int64_t rb = blocks8(q.rows), cb = blocks8(q.cols);
  for_dtype(w.dtype, [&](auto type) {
    using T = decltype(type);
    const bool whole = on_16(w.data, w.row_stride, w.dtype, w.group_stride);
    launch_next(k_dequantise_weights<T>, dim3(static_cast<unsigned>(q.groups * rb * cb)), kThreads, 0, s, bytes(q.values),
                q.group_stride, q.row_stride, q.scales, q.rows, q.cols, rb, cb, static_cast<T*>(w.data), w.group_stride,
                w.row_stride, whole);
  });
}

void launch_gated8(const spgemm_dense& pre, const spgemm_dense& h, const spgemm_rows8& gate, const spgemm_rows8& up,
                   cudaStream_t s) {
  const int64_t hidden = h.cols;
  if (pre.rows == 0 || hidden == 0) return;
  for_dtype(pre.dtype, [&](auto type) {
    for_dtype(h.dtype, [&](auto out) {
      using T = decltype(type);
      using TO = decltype(out);
      launch_next(k_gated8<T, TO>, row_grid(pre.rows, hidden), kThreads, 0, s, static_cast<const T*>(pre.data), pre.stride,
                  on_16(pre.data, pre.stride, pre.dtype), on_16(pre.data, pre.stride, pre.dtype, hidden), pre.rows, hidden,
                  static_cast<TO*>(h.data), h.stride, on_16(h.data, h.stride, h.dtype), bytes(gate.values), gate.stride,
                  gate.scales, gate.scale_stride, bytes(up.values), up.stride, up.scales, up.scale_stride);
    });
  });
}

void launch_gated8_backward(const spgemm_dense& dh, const spgemm_rows8& gate, const spgemm_rows8& up, const spgemm_dense& dpre,
                            const spgemm_dense* h, cudaStream_t s) {
  const int64_t hidden = dh.cols;
  if (dh.rows == 0 || hidden == 0) return;
  for_dtype(dh.dtype, [&](auto type) {
    using T = decltype(type);
    launch_next(k_gated8_backward<T>, row_grid(dh.rows, hidden), kThreads, 0, s, static_cast<const T*>(dh.data), dh.stride,
                on_16(dh.data, dh.stride, dh.dtype), dh.rows, hidden, bytes(gate.values), gate.stride, gate.scales,
                gate.scale_stride, bytes(up.values), up.stride, up.scales, up.scale_stride, static_cast<T*>(dpre.data), dpre.stride,
                on_16(dpre.data, dpre.stride, dpre.dtype), on_16(dpre.data, dpre.stride, dpre.dtype, hidden),
                static_cast<T*>(h ? h->data : nullptr), h ? h->stride : 0, h && on_16(h->data, h->stride, h->dtype));
  });
}

}  // namespace sg
