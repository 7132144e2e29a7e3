// Internal interface of the grouped-product operators (routing, expert products, adapters).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace sg {

constexpr int kMaxGroups = 1024;   // experts or adapters of one call
constexpr int kMaxTopK = 32;       // slots of one token

// Device error word of the grouped operators (spgemm_grouped_status reads and clears it).
uint32_t* grouped_err();

// ---- element conversions -------------------------------------------------------------------
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// silu(g) * u in 32 bits.  exp overflows to +inf for g below -88: g / inf = -0, the limit.
__device__ __forceinline__ float gated_silu(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// Launches of one call follow each other without a gap: a kernel may be started while the one before it
// ends.  Every kernel launched this way calls pdl_wait before its first access to global memory (it
// returns when everything before it on the stream is complete and visible), and pdl_go once to let
// the next one start.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
inline bool launch_next(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...) == cudaSuccess;
}

// The same for a result that is rounded to 16 bits: relative error below 2^-18 for |g| < 60, below
// which silu is smaller than any f16 and than 2^-80.
__device__ __forceinline__ float gated_silu_short(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

inline int dtype_size(int32_t d) { return d == SPGEMM_DTYPE_F32 ? 4 : 2; }

template <typename F>
inline void for_dtype(int32_t d, F f) {
  if (d == SPGEMM_DTYPE_F32) f(float());
  else if (d == SPGEMM_DTYPE_BF16) f(__nv_bfloat16());
  else f(__half());
}

// ---- routing (k_route.cu) ------------------------------------------------------------------
struct RouteOut {
  int32_t* ids;
  float* weights;
  int32_t *offsets, *order, *position;
};
// bytes of device scratch the two transposing calls need (0: none)
int64_t route_scratch_bytes(int64_t tokens, int32_t experts);
int64_t group_scratch_bytes(int64_t slots, int32_t groups);
void launch_route(const spgemm_dense& logits, const spgemm_route_rule& rule, const float* bias, const RouteOut& out,
                  void* scratch, cudaStream_t s);
void launch_route_backward(const spgemm_dense& logits, const spgemm_route_rule& rule, const int32_t* ids,
                           const float* grad_w, const spgemm_dense& out, cudaStream_t s);
void launch_group_rows(const int32_t* ids, int64_t slots, int32_t groups, int32_t* offsets, int32_t* order,
                       int32_t* position, void* scratch, cudaStream_t s);

// ---- weighted sums over a token's slots (k_combine.cu) --------------------------------------
// out[t] = sum_j w[t,j] * y[position[t,j]]; weights NULL: all ones
void launch_combine(const spgemm_grouping& g, const float* weights, const spgemm_dense& y, const spgemm_dense& out,
                    cudaStream_t s);
void launch_combine_backward(const spgemm_grouping& g, const float* weights, const spgemm_dense& dout,
                             const spgemm_dense& y, const spgemm_dense& dy, float* dweights, cudaStream_t s);

// out[position of slot] = x[slot's token] for every slot with a group (16-bit, 16-byte aligned rows);
// rows of out behind the last group are not written
void launch_spread_rows(const spgemm_grouping& g, const spgemm_dense& x, const spgemm_dense& out, cudaStream_t s);

// ---- grouped products on CUDA cores, any type, stride and alignment (k_group_plain.cu) --------
// y[p, :] = x[row(p), :] * w[g]^T for every position p of group g; row(p) = order[p] / top_k when
// gather, else p; rows of y past the last group are set to zero.  y may be 32-bit.
void launch_plain_forward(const spgemm_grouping& g, const spgemm_dense& x, bool gather, const spgemm_weights& w,
                          const spgemm_dense& y, cudaStream_t s);
// dx[p, :] = dy[p, :] * w[g] (32-bit, one row per position)
void launch_plain_dx(const spgemm_grouping& g, const spgemm_dense& dy, const spgemm_weights& w, float* dx,
                     cudaStream_t s);
// dw[g] = sum over the group's positions of dy[p, :]^T x[row(p), :]
void launch_plain_dw(const spgemm_grouping& g, const spgemm_dense& dy, const spgemm_dense& x,
                     const spgemm_weights& dw, cudaStream_t s);
// h[p, i] = silu(pre[p, i]) * pre[p, hidden + i]
void launch_gated(const float* pre, int64_t rows, int64_t hidden, const spgemm_dense& h, cudaStream_t s);
// y[t, :] = base[t, :] + scale[id] * v[position[t], :] * b[id]^T (base, v: 32-bit)
void launch_plain_adapter_add(const spgemm_grouping& g, const int32_t* ids, const float* scale, const float* base,
                              const float* v, int64_t rank, const spgemm_weights& b, const spgemm_dense& y,
                              cudaStream_t s);

}  // namespace sg
