// Routing: router logits -> the chosen experts of every token, their weights, and the choice
// transposed (the slots in order of their expert); the gradient of the logits; the transpose of
// given ids.
//
//   s = softmax(l) or 1 / (1 + exp(-l));  c = s + bias, or l itself without a bias (both scores
//   rise with l, so comparing l is the same choice without its rounding);  the k largest c among
//   the kept expert groups;  w = s / sum of the chosen s * scale.
//
// One warp per token: lane i holds experts i, i + 32, ... in registers, so a row is read once,
// coalesced, and softmax, group scores and the k rounds of "largest remaining" are warp
// reductions.  A float is compared through an integer with the same order, which makes each
// round two warp-wide integer reductions (largest key, then lowest index that has it).
// The chosen experts leave in ascending order for free: ballots over the register index.
//
// The transpose is a stable counting sort.  Each warp owns consecutive tokens and counts per
// expert in its own row of shared memory; the count before the increment is the slot's rank in
// the warp (the experts of one token differ, so no two lanes meet).  The block adds its warps up
// and writes its counts; k_block_offsets scans them over the blocks, k_group_scatter over the experts.
// Sums of ranks and scans are integers: the result does not depend on the order of the blocks.
#include <algorithm>

#include "groups.h"

namespace sg {

namespace {

constexpr int kWarps = 8;              // warps of a block
constexpr int kTokensPerWarp = 8;      // consecutive tokens of a warp (route)
constexpr int kSlotsPerWarp = 256;     // consecutive slots of a warp (given ids)
constexpr float kNegInf = -INFINITY;

// An unsigned integer with the order of the floats; 0 is kept for "not selectable".
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 compares equal to +0
  return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float warp_max_f(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}

// A row of logits into registers (element v of lane i is expert 32 v + i), then its scores.
template <typename T, int NV>
__device__ __forceinline__ void row_scores(const T* __restrict__ row, int experts, int score, float (&l)[NV],
                                           float (&s)[NV]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = v * 32 + lane;
    float x = e < experts ? to_f32(row[e]) : kNegInf;
    x = x != x ? kNegInf : fminf(x, 3.402823466e+38f);
    l[v] = x;
  }
  if (score == SPGEMM_SCORE_SIGMOID) {
#pragma unroll
    for (int v = 0; v < NV; ++v) s[v] = 1.0f / (1.0f + expf(-l[v]));
    return;
  }
  float top = l[0];
#pragma unroll
  for (int v = 1; v < NV; ++v) top = fmaxf(top, l[v]);
  top = warp_max_f(top);
  float sum = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    s[v] = l[v] > kNegInf ? expf(l[v] - top) : 0.0f;
    sum += s[v];
  }
  sum = warp_sum(sum);
#pragma unroll
  for (int v = 0; v < NV; ++v) s[v] = sum > 0.0f ? s[v] / sum : 0.0f;
}

// Clears the keys of the expert groups that are not kept.
template <int NV>
__device__ __forceinline__ void keep_groups(const spgemm_route_rule& r, int experts, bool by_scores, const float (&s)[NV],
                                            uint32_t (&key)[NV]) {
  const int lane = threadIdx.x & 31;
  const int per = experts / r.groups;
  float mine = kNegInf;  // lane g: the score of group g
  for (int g = 0; g < r.groups; ++g) {
    uint32_t best = 0, second = 0;
    int at = 0x7fffffff;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = v * 32 + lane;
      if (e / per != g || e >= experts || key[v] == 0) continue;
      const uint32_t k = by_scores ? order_key(s[v]) : key[v];
      if (k > best) {
        second = best;
        best = k;
        at = e;
      } else if (k > second) {
        second = k;
      }
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    float val = top ? key_value(top) : kNegInf;
    if (r.group_score == SPGEMM_GROUP_TOP2 && top) {
      const int first = static_cast<int>(
          __reduce_min_sync(0xffffffffu, best == top ? static_cast<uint32_t>(at) : 0xffffffffu));
      const uint32_t next = __reduce_max_sync(0xffffffffu, (best == top && at == first) ? second : best);
      if (next) val += key_value(next);
    }
    if (lane == g) mine = val;
  }
  int rank = 0;
  for (int g = 0; g < r.groups; ++g) {
    const float o = __shfl_sync(0xffffffffu, mine, g);
    if (o > mine || (o == mine && g < lane)) ++rank;
  }
  const uint32_t kept = __ballot_sync(0xffffffffu, lane < r.groups && rank < r.groups_kept);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = v * 32 + lane;
    if (e < experts && !((kept >> (e / per)) & 1u)) key[v] = 0;
  }
}

// The choice of one token; writes ids and weights of its row and, with `rank`, the rank of each
// slot among the warp's earlier slots of the same expert (counted in cnt[experts]).
template <typename T, int NV>
__device__ __forceinline__ void route_token(const T* __restrict__ row, int experts, const spgemm_route_rule& r,
                                            const float* __restrict__ bias, int32_t* __restrict__ ids,
                                            float* __restrict__ weights, int32_t* __restrict__ rank, int* cnt) {
  const int lane = threadIdx.x & 31;
  float l[NV], s[NV];
  row_scores<T, NV>(row, experts, r.score, l, s);
  uint32_t key[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = v * 32 + lane;
    const float c = bias && e < experts ? s[v] + bias[e] : l[v];
    key[v] = l[v] > kNegInf && c > kNegInf ? order_key(c) : 0u;
  }
  if (r.groups_kept < r.groups)
    keep_groups<NV>(r, experts, !bias && r.group_score == SPGEMM_GROUP_TOP2, s, key);
  uint32_t chosen = 0;  // bit v: expert 32 v + lane
  uint32_t best = 0;
  int at = 0;
  bool stale = true;
  for (int j = 0; j < r.top_k; ++j) {
    if (stale) {  // only the lane whose expert was taken looks again
      best = 0;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (key[v] > best) {
          best = key[v];
          at = v;
        }
      stale = false;
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    if (top == 0) break;
    const uint32_t e = __reduce_min_sync(0xffffffffu, best == top ? static_cast<uint32_t>(at * 32 + lane) : 0xffffffffu);
    if ((e & 31u) == static_cast<uint32_t>(lane)) {
      chosen |= 1u << at;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v == at) key[v] = 0;
      stale = true;
    }
  }
  float f = r.scale;
  if (r.renormalise) {
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if ((chosen >> v) & 1u) sum += s[v];
    sum = warp_sum(sum);
#pragma unroll
    for (int v = 0; v < NV; ++v) s[v] = sum > 0.0f ? s[v] / sum : 0.0f;
  }
  int n = 0;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const bool c = (chosen >> v) & 1u;
    const uint32_t b = __ballot_sync(0xffffffffu, c);
    if (c) {
      const int j = n + __popc(b & lanemask_lt());
      const int e = v * 32 + lane;
      ids[j] = e;
      weights[j] = s[v] * f;
      rank[j] = cnt[e]++;
    }
    n += __popc(b);
  }
  if (lane >= n && lane < r.top_k) {
    ids[lane] = -1;
    weights[lane] = 0.0f;
    rank[lane] = -1;
  }
}

// cnt[w * groups + e] (counts of warp w) -> exclusive prefix over the warps; total[e] = block sum.
__device__ __forceinline__ void warp_prefix(int* cnt, int groups, int32_t* total) {
  for (int e = threadIdx.x; e < groups; e += blockDim.x) {
    int sum = 0;
    for (int w = 0; w < kWarps; ++w) {
      const int c = cnt[w * groups + e];
      cnt[w * groups + e] = sum;
      sum += c;
    }
    total[e] = sum;
  }
}

}  // namespace

// ids, weights; position[slot] = the slot's rank among the block's slots of the same expert;
// counts[block * experts + e] = the block's slots of expert e.
template <typename T, int NV>
__global__ void __launch_bounds__(kWarps * 32) k_route(const T* __restrict__ logits, int64_t stride, int64_t tokens,
                                                       int experts, spgemm_route_rule r,
                                                       const float* __restrict__ bias, int32_t* __restrict__ ids,
                                                       float* __restrict__ weights, int32_t* __restrict__ position,
                                                       int32_t* __restrict__ counts) {
  extern __shared__ int s_cnt[];  // kWarps x experts
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kWarps * experts; i += blockDim.x) s_cnt[i] = 0;
  __syncthreads();
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kTokensPerWarp;
  const int64_t t1 = min(tokens, t0 + kTokensPerWarp);
  for (int64_t t = t0; t < t1; ++t) {
    const int64_t o = t * r.top_k;
    route_token<T, NV>(logits + t * stride, experts, r, bias, ids + o, weights + o, position + o,
                       s_cnt + warp * experts);
    __syncwarp();
  }
  __syncthreads();
  warp_prefix(s_cnt, experts, counts + static_cast<int64_t>(blockIdx.x) * experts);
  __syncthreads();
  for (int64_t i = t0 * r.top_k + lane; i < t1 * r.top_k; i += 32) {
    const int e = ids[i];
    if (e >= 0) position[i] += s_cnt[warp * experts + e];
  }
}

// The same counts and ranks for given ids: equal ids among 32 consecutive slots are ranked by a
// warp match.
__global__ void __launch_bounds__(kWarps * 32) k_count_ids(const int32_t* __restrict__ ids, int64_t slots, int groups,
                                                           int32_t* __restrict__ position, int32_t* __restrict__ counts,
                                                           uint32_t* err) {
  extern __shared__ int s_cnt[];  // kWarps x groups
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kWarps * groups; i += blockDim.x) s_cnt[i] = 0;
  __syncthreads();
  int* cnt = s_cnt + warp * groups;
  const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kSlotsPerWarp;
  const int64_t i1 = min(slots, i0 + kSlotsPerWarp);
  for (int64_t b = i0; b < i1; b += 32) {
    const int64_t i = b + lane;
    int e = i < i1 ? ids[i] : -1;
    if (e >= groups || e < -1) {
      set_error(err, kErrBounds);
      e = -1;
    }
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const int before = __popc(same & lanemask_lt());
    const int base = e >= 0 ? cnt[e] : 0;
    __syncwarp();
    if (e >= 0 && before == 0) cnt[e] = base + __popc(same);
    __syncwarp();
    if (i < i1) position[i] = e >= 0 ? base + before : -1;
  }
  __syncthreads();
  warp_prefix(s_cnt, groups, counts + static_cast<int64_t>(blockIdx.x) * groups);
  __syncthreads();
  for (int64_t i = i0 + lane; i < i1; i += 32)
    if (position[i] >= 0) position[i] += cnt[ids[i]];
}

// counts[b * groups + e] -> the slots of group e in the blocks before b; total[e] = all of them.
// One warp per group.
__global__ void __launch_bounds__(kWarps * 32) k_block_offsets(int32_t* __restrict__ counts, int64_t blocks, int groups,
                                                               int32_t* __restrict__ total) {
  const int e = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (e >= groups) return;
  int run = 0;
  for (int64_t b0 = 0; b0 < blocks; b0 += 32) {
    const int64_t b = b0 + lane;
    const int c = b < blocks ? counts[b * groups + e] : 0;
    const int incl = warp_incl_scan(c);
    if (b < blocks) counts[b * groups + e] = run + incl - c;
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) total[e] = run;
}

// position: rank in the block -> position; order: its inverse; offsets.  per_block consecutive
// slots belong to one block of the counting kernel, and to one block here.
__global__ void __launch_bounds__(kWarps * 32) k_group_scatter(const int32_t* __restrict__ ids, int64_t slots,
                                                               int64_t per_block, int groups,
                                                               const int32_t* __restrict__ counts,
                                                               const int32_t* __restrict__ total,
                                                               int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                                                               int32_t* __restrict__ position) {
  extern __shared__ int s_off[];  // groups + 1
  __shared__ int s_tmp[33];
  int run = 0;
  for (int e0 = 0; e0 < groups; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    const int c = e < groups ? total[e] : 0;
    int sum;
    const int incl = block_incl_scan(c, s_tmp, &sum);
    if (e < groups) s_off[e] = run + incl - c;
    run += sum;
  }
  if (threadIdx.x == 0) s_off[groups] = run;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= groups; e += blockDim.x) offsets[e] = s_off[e];
  const int32_t* base = counts + static_cast<int64_t>(blockIdx.x) * groups;
  const int64_t i1 = min(slots, (static_cast<int64_t>(blockIdx.x) + 1) * per_block);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x; i < i1; i += blockDim.x) {
    const int r = position[i];
    if (r >= 0) {
      const int e = ids[i];
      const int p = s_off[e] + base[e] + r;
      position[i] = p;
      order[p] = static_cast<int32_t>(i);
    }
    if (i >= run) order[i] = -1;  // positions behind the last group
  }
}

// Gradient of the logits.  One warp per token; the row's scores are computed again.
template <typename T, int NV>
__global__ void __launch_bounds__(kWarps * 32) k_route_backward(const T* __restrict__ logits, int64_t stride,
                                                                int64_t tokens, int experts, spgemm_route_rule r,
                                                                const int32_t* __restrict__ ids,
                                                                const float* __restrict__ grad_w, T* __restrict__ out,
                                                                int64_t out_stride) {
  __shared__ float s_row[kWarps][kMaxGroups > NV * 32 ? NV * 32 : kMaxGroups];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* full = s_row[warp];  // scores, then gradients of the scores, of the whole row
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < tokens;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    float l[NV], s[NV];
    row_scores<T, NV>(logits + t * stride, experts, r.score, l, s);
    int e = lane < r.top_k ? ids[t * r.top_k + lane] : -1;
    if (e >= experts) e = -1;
    float ds = e >= 0 ? grad_w[t * r.top_k + lane] * r.scale : 0.0f;
    if (r.renormalise) {  // w = s / sum: ds = (dw - sum of dw * w) / sum
#pragma unroll
      for (int v = 0; v < NV; ++v) full[v * 32 + lane] = s[v];
      __syncwarp();
      const float mine = e >= 0 ? full[e] : 0.0f;
      const float sum = warp_sum(mine);
      const float dot = sum > 0.0f ? warp_sum(ds * (mine / sum)) : 0.0f;
      ds = e >= 0 && sum > 0.0f ? (ds - dot) / sum : 0.0f;
      __syncwarp();
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) full[v * 32 + lane] = 0.0f;
    __syncwarp();
    if (e >= 0) full[e] = ds;
    __syncwarp();
    float dot = 0.0f;
    if (r.score == SPGEMM_SCORE_SOFTMAX) {
#pragma unroll
      for (int v = 0; v < NV; ++v) dot += full[v * 32 + lane] * s[v];
      dot = warp_sum(dot);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = v * 32 + lane;
      const float d = full[i];
      const float g = r.score == SPGEMM_SCORE_SOFTMAX ? s[v] * (d - dot) : d * s[v] * (1.0f - s[v]);
      if (i < experts) out[t * out_stride + i] = from_f32<T>(g);
    }
    __syncwarp();
  }
}

namespace {

// f(integral constant NV) for the smallest number of registers per lane that holds a row
template <typename F>
void for_width(int experts, F f) {
  if (experts <= 32) f(std::integral_constant<int, 1>());
  else if (experts <= 64) f(std::integral_constant<int, 2>());
  else if (experts <= 128) f(std::integral_constant<int, 4>());
  else if (experts <= 256) f(std::integral_constant<int, 8>());
  else if (experts <= 512) f(std::integral_constant<int, 16>());
  else f(std::integral_constant<int, 32>());
}

int64_t scratch_bytes(int64_t blocks, int64_t groups) { return 4 * (blocks * groups + groups); }

void transpose(const int32_t* ids, int64_t slots, int64_t per_block, int64_t blocks, int groups, int32_t* counts,
               int32_t* offsets, int32_t* order, int32_t* position, cudaStream_t s) {
  int32_t* total = counts + blocks * groups;
  note_launch();
  k_block_offsets<<<static_cast<unsigned>(ceil_div(groups, kWarps)), kWarps * 32, 0, s>>>(counts, blocks, groups, total);
  note_launch();
  k_group_scatter<<<static_cast<unsigned>(std::max<int64_t>(blocks, 1)), kWarps * 32, sizeof(int) * (groups + 1), s>>>(
      ids, slots, per_block, groups, counts, total, offsets, order, position);
}

}  // namespace

int64_t route_scratch_bytes(int64_t tokens, int32_t experts) {
  return scratch_bytes(ceil_div(tokens, kWarps * kTokensPerWarp), experts);
}
int64_t group_scratch_bytes(int64_t slots, int32_t groups) {
  return scratch_bytes(ceil_div(slots, kWarps * kSlotsPerWarp), groups);
}

void launch_route(const spgemm_dense& logits, const spgemm_route_rule& rule, const float* bias, const RouteOut& out,
                  void* scratch, cudaStream_t s) {
  const int64_t tokens = logits.rows;
  const int experts = static_cast<int>(logits.cols);
  int32_t* counts = static_cast<int32_t*>(scratch);
  const int64_t blocks = ceil_div(tokens, kWarps * kTokensPerWarp);
  if (blocks > 0)
    for_dtype(logits.dtype, [&](auto type) {
      for_width(experts, [&](auto nv) {
        using T = decltype(type);
        note_launch();
        k_route<T, nv.value><<<static_cast<unsigned>(blocks), kWarps * 32, sizeof(int) * kWarps * experts, s>>>(
            static_cast<const T*>(logits.data), logits.stride, tokens, experts, rule, bias, out.ids, out.weights,
            out.position, counts);
      });
    });
  transpose(out.ids, tokens * rule.top_k, static_cast<int64_t>(kWarps) * kTokensPerWarp * rule.top_k, blocks, experts,
            counts, out.offsets, out.order, out.position, s);
}

void launch_group_rows(const int32_t* ids, int64_t slots, int32_t groups, int32_t* offsets, int32_t* order,
                       int32_t* position, void* scratch, cudaStream_t s) {
  int32_t* counts = static_cast<int32_t*>(scratch);
  const int64_t blocks = ceil_div(slots, kWarps * kSlotsPerWarp);
  if (blocks > 0) {
    note_launch();
    k_count_ids<<<static_cast<unsigned>(blocks), kWarps * 32, sizeof(int) * kWarps * groups, s>>>(
        ids, slots, groups, position, counts, grouped_err());
  }
  transpose(ids, slots, static_cast<int64_t>(kWarps) * kSlotsPerWarp, blocks, groups, counts, offsets, order, position,
            s);
}

void launch_route_backward(const spgemm_dense& logits, const spgemm_route_rule& rule, const int32_t* ids,
                           const float* grad_w, const spgemm_dense& out, cudaStream_t s) {
  const int64_t tokens = logits.rows;
  const int experts = static_cast<int>(logits.cols);
  if (tokens == 0) return;
  const int64_t blocks = std::min<int64_t>(ceil_div(tokens, kWarps), 1 << 20);
  for_dtype(logits.dtype, [&](auto type) {
    for_width(experts, [&](auto nv) {
      using T = decltype(type);
      note_launch();
      k_route_backward<T, nv.value><<<static_cast<unsigned>(blocks), kWarps * 32, 0, s>>>(
          static_cast<const T*>(logits.data), logits.stride, tokens, experts, rule, ids, grad_w,
          static_cast<T*>(out.data), out.stride);
    });
  });
}

}  // namespace sg
