// Routing: router logits -> the chosen experts of every token, their weights, and the choice
// transposed (the slots in order of their expert); the gradient of the logits; the transpose of
// given ids.
//
//   s = softmax(l) or 1 / (1 + exp(-l));  c = s + bias, or l itself without a bias (both scores
//   rise with l, so comparing l is the same choice without its rounding);  the k largest c among
//   the kept expert groups;  w = s / sum of the chosen s * scale.
//
// L lanes hold a token's row, V consecutive experts each (8 lanes x 8 up to 64 experts, 16 x 8, 32 x 8,
// then 32 x 16 and 32 x 32): a row is read once in 16-byte pieces, and a warp works on 32 / L tokens at
// once, which is what a router is bound by: instructions, not bytes.  A float is compared through an
// integer with the same order; each round of "largest remaining" is a maximum over the L lanes and a
// ballot, whose lowest set bit is the lowest index because lanes hold consecutive experts.  For the same
// reason the chosen experts leave in ascending order after one prefix sum of their counts.
//
// The transpose is a stable counting sort.  Each warp owns consecutive tokens and counts per
// expert in its own row of shared memory, its tokens one after the other: the count before a slot is
// its rank in the warp.  The block adds its
// warps up and writes its counts; k_block_offsets scans them over the blocks, k_group_scatter
// over the experts.  Few tokens (one block's worth) finish in the first kernel.
// Ranks and scans are integers: the result does not depend on the order of the blocks.
//
// Measured on GB300: 16 x 64 (32-bit logits) 7 us in one launch, latency; 16384 x 256 (32-bit, sigmoid, bias,
// 8 groups) 34 us + 12 us for the transpose, 17 MB read at 0.5 TB/s; 65536 x 64 (bf16) 29 us + 13 us.  Both
// are bound by instructions: 70% of the issue slots, about 1050 warp instructions per 256-expert row and
// 1400 per four 64-expert rows.  (One warp per token: 115 and 43 us.)
#include <algorithm>

#include "groups.h"

namespace sg {

namespace {

constexpr int kWarps = 8;               // warps of a block
constexpr int kWarpsOne = 32;           // of the block that does everything
constexpr int kSteps = 2;               // most steps (32 / L tokens each) of a warp of many blocks
constexpr int kSlotsPerWarp = 64;       // consecutive slots of a warp (given ids), of one block or many
constexpr int kOneExperts = 256;        // most experts whose counts the single block keeps (32 KB, what needs no opt-in)
constexpr float kNegInf = -INFINITY;

// An unsigned integer with the order of the floats; 0 is kept for "not selectable".
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 compares equal to +0
  return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if (L == 32) return __reduce_max_sync(0xffffffffu, v);
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_max_f(float v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}
// the lanes of this token in a ballot
template <int L>
__device__ __forceinline__ uint32_t lanes_of(uint32_t ballot) {
  return L == 32 ? ballot : (ballot >> (lane_id() & ~(L - 1))) & ((1u << (L & 31)) - 1u);
}

template <typename T, int V>
struct alignas(sizeof(T) * V > 16 ? 16 : sizeof(T) * V) Piece {
  T v[V];
};

// A row of logits into registers (element v of the token's lane i is expert i V + v).  `row` NULL: no token.
template <typename T, int L, int V>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int experts, bool pieces, float (&l)[V]) {
  const int e0 = (lane_id() & (L - 1)) * V;
  if (row && pieces && e0 + V <= experts) {
    const Piece<T, V> p = *reinterpret_cast<const Piece<T, V>*>(row + e0);
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = to_f32(p.v[v]);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = row && e0 + v < experts ? to_f32(row[e0 + v]) : kNegInf;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = l[v] != l[v] ? kNegInf : fminf(l[v], 3.402823466e+38f);
}

// Scores of a row are s[v] * (the returned factor): softmax's division by the sum is left to the few
// values that need it.
template <int L, int V>
__device__ __forceinline__ float row_scores(int score, const float (&l)[V], float (&s)[V]) {
  if (score == SPGEMM_SCORE_SIGMOID) {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = 1.0f / (1.0f + expf(-l[v]));
    return 1.0f;
  }
  float top = l[0];
#pragma unroll
  for (int v = 1; v < V; ++v) top = fmaxf(top, l[v]);
  top = lanes_max_f<L>(top);
  float sum = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s[v] = l[v] > kNegInf ? expf(l[v] - top) : 0.0f;
    sum += s[v];
  }
  sum = lanes_sum<L>(sum);
  return sum > 0.0f ? 1.0f / sum : 0.0f;
}

// best and second of two pairs (second may equal best)
__device__ __forceinline__ void merge_two(uint32_t& best, uint32_t& second, uint32_t b, uint32_t s) {
  second = max(min(best, b), max(second, s));
  best = max(best, b);
}

// Clears the keys of the expert groups that are not kept.  `val`: 32 floats of this token.
template <int L, int V>
__device__ __forceinline__ void keep_groups(const spgemm_route_rule& r, int per, bool by_scores, const float (&s)[V],
                                            uint32_t (&key)[V], float* val) {
  const int me = lane_id() & (L - 1), e0 = me * V;
  const bool top2 = r.group_score == SPGEMM_GROUP_TOP2;
  auto score_of = [&](uint32_t best, uint32_t second) {
    float f = best ? key_value(best) : kNegInf;
    if (top2 && second) f += key_value(second);
    return f;
  };
  const int wide = per / V;  // lanes of a group, when groups are whole lanes
  if (per % V == 0 && (wide & (wide - 1)) == 0 && wide <= L) {
    uint32_t best = 0, second = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t k = key[v] == 0 ? 0u : by_scores ? order_key(s[v]) : key[v];
      merge_two(best, second, k, 0u);
    }
    for (int d = 1; d < wide; d <<= 1)
      merge_two(best, second, __shfl_xor_sync(0xffffffffu, best, d), __shfl_xor_sync(0xffffffffu, second, d));
    if (me % wide == 0 && e0 / per < r.groups) val[e0 / per] = score_of(best, second);
  } else {
    for (int g = 0; g < r.groups; ++g) {
      uint32_t best = 0, second = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const bool in = e0 + v >= g * per && e0 + v < (g + 1) * per && key[v] != 0;
        const uint32_t k = !in ? 0u : by_scores ? order_key(s[v]) : key[v];
        merge_two(best, second, k, 0u);
      }
#pragma unroll
      for (int d = 1; d < L; d <<= 1)
        merge_two(best, second, __shfl_xor_sync(0xffffffffu, best, d), __shfl_xor_sync(0xffffffffu, second, d));
      if (me == 0) val[g] = score_of(best, second);
    }
  }
  __syncwarp();
  uint32_t kept = 0;
  for (int g = me; g < r.groups; g += L) {
    const float mine = val[g];
    int rank = 0;
    for (int o = 0; o < r.groups; ++o) rank += val[o] > mine || (val[o] == mine && o < g) ? 1 : 0;
    if (rank < r.groups_kept) kept |= 1u << g;
  }
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) kept |= __shfl_xor_sync(0xffffffffu, kept, d);
  int g = e0 / per, left = (g + 1) * per - e0;  // group of expert e0 + v, and experts of it still to come
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!((kept >> (g & 31)) & 1u)) key[v] = 0;
    if (--left == 0) {
      ++g;
      left = per;
    }
  }
  __syncwarp();
}

// cnt[w * groups + e] (counts of warp w) -> exclusive prefix over the warps; the sum of e.
__device__ __forceinline__ int warp_prefix(int* cnt, int groups, int warps, int e) {
  int sum = 0;
  for (int w = 0; w < warps; ++w) {
    const int c = cnt[w * groups + e];
    cnt[w * groups + e] = sum;
    sum += c;
  }
  return sum;
}

// s_off[e] = first position of group e from its total (`of(e)`); returns the sum.  All threads call it.
template <typename F>
__device__ __forceinline__ int group_offsets(int groups, int* s_off, int* s_tmp, F of) {
  int run = 0;
  for (int e0 = 0; e0 < groups; e0 += blockDim.x) {
    const int e = e0 + static_cast<int>(threadIdx.x);
    const int c = e < groups ? of(e) : 0;
    int sum;
    const int incl = block_incl_scan(c, s_tmp, &sum);
    if (e < groups) s_off[e] = run + incl - c;
    run += sum;
  }
  if (threadIdx.x == 0) s_off[groups] = run;
  __syncthreads();
  return run;
}

}  // namespace

// ids and weights.  ONE: also offsets, order and position (one block).  Otherwise position[slot] = the
// slot's rank among the block's slots of the same expert and counts[e * blocks + block] = the block's
// slots of expert e.
template <typename T, int L, int V, bool ONE>
__global__ void __launch_bounds__((ONE ? kWarpsOne : kWarps) * 32, ONE || V > 8 ? 1 : 4)
    k_route(const T* __restrict__ logits, int64_t stride, int64_t tokens, int experts, int pieces, int steps,
            const __grid_constant__ spgemm_route_rule r, const float* __restrict__ bias, int32_t* __restrict__ ids,
            float* __restrict__ weights, int32_t* __restrict__ position, int32_t* __restrict__ counts,
            int32_t* __restrict__ offsets, int32_t* __restrict__ order) {
  constexpr int kW = ONE ? kWarpsOne : kWarps, kPer = 32 / L;
  extern __shared__ int s_cnt[];  // kW x experts, then (ONE) experts + 1 offsets
  __shared__ float s_val[kW][kPer][32];
  __shared__ int s_tmp[33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int me = lane & (L - 1), sub = lane / L, e0 = me * V;
  pdl_wait();
  pdl_go();
  for (int i = threadIdx.x; i < kW * experts; i += blockDim.x) s_cnt[i] = 0;
  __syncthreads();
  int* cnt = s_cnt + warp * experts;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kW + warp) * (steps * kPer);
  const int64_t t1 = min(tokens, t0 + steps * kPer);
  const int per = experts / r.groups;
  float mine_bias[V];
#pragma unroll
  for (int v = 0; v < V; ++v) mine_bias[v] = bias && e0 + v < experts ? bias[e0 + v] : 0.0f;
  for (int64_t tw = t0; tw < t1; tw += kPer) {
    const int64_t t = tw + sub;
    const bool there = t < t1;
    float l[V], s[V];
    load_row<T, L, V>(there ? logits + t * stride : nullptr, experts, pieces, l);
    float f = row_scores<L, V>(r.score, l, s);
    if (bias || r.group_score == SPGEMM_GROUP_TOP2) {  // scores are compared or added: they want their division
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] *= f;
      f = 1.0f;
    }
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float c = bias ? s[v] + mine_bias[v] : l[v];
      key[v] = l[v] > kNegInf && c > kNegInf ? order_key(c) : 0u;
    }
    if (r.groups_kept < r.groups)
      keep_groups<L, V>(r, per, !bias && r.group_score == SPGEMM_GROUP_TOP2, s, key, s_val[warp][sub]);
    uint32_t chosen = 0;  // bit v: expert e0 + v
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (key[v] > best) {
        best = key[v];
        at = v;
      }
    for (int j = 0; j < r.top_k; ++j) {
      const uint32_t top = lanes_max<L>(best);
      const uint32_t have = lanes_of<L>(__ballot_sync(0xffffffffu, best == top && top != 0));
      if (have && __ffs(have) - 1 == me) {  // this lane's expert is taken: look for its next best
        chosen |= 1u << at;
        best = 0;
        const int was = at;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (v == was) key[v] = 0;
          if (key[v] > best) {
            best = key[v];
            at = v;
          }
        }
      }
    }
    float over = 1.0f;  // a division per chosen expert: a single one has the weight 1 exactly
    if (r.renormalise) {
      float sum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if ((chosen >> v) & 1u) sum += s[v];
      sum = lanes_sum<L>(sum);
      f = sum > 0.0f ? 1.0f : 0.0f;  // the row's own factor cancels
      over = sum > 0.0f ? sum : 1.0f;
    }
    f *= r.scale;
    int before = __popc(chosen);  // chosen experts of the lower lanes
    const int mine = before;
#pragma unroll
    for (int d = 1; d < L; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, before, d, L);
      if (me >= d) before += o;
    }
    const int n = __shfl_sync(0xffffffffu, before, L - 1, L);
    int64_t o = t * r.top_k + before - mine;
    // tokens of a step take their ranks one after the other; a lane has few chosen experts
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      if (kPer == 1 || sub == q)
        for (uint32_t left = chosen; left; left &= left - 1, ++o) {
          const int v = __ffs(left) - 1;
          float w = 0.0f;
#pragma unroll
          for (int i = 0; i < V; ++i) w = i == v ? s[i] : w;
          const int rank = cnt[e0 + v]++;
          ids[o] = e0 + v;
          weights[o] = w / over * f;
          position[o] = rank;
        }
      if (kPer > 1) __syncwarp();
    }
    for (int j = n + me; there && j < r.top_k; j += L) {
      ids[t * r.top_k + j] = -1;
      weights[t * r.top_k + j] = 0.0f;
      position[t * r.top_k + j] = -1;
    }
    __syncwarp();
  }
  __syncthreads();
  const int64_t i0 = t0 * r.top_k + lane, i1 = t1 * r.top_k;
  if (!ONE) {
    for (int e = threadIdx.x; e < experts; e += blockDim.x)
      counts[static_cast<int64_t>(e) * gridDim.x + blockIdx.x] = warp_prefix(s_cnt, experts, kW, e);
    __syncthreads();
    for (int64_t i = i0; i < i1; i += 32) {
      const int e = ids[i];
      if (e >= 0) position[i] += cnt[e];
    }
  } else {
    int* s_off = s_cnt + kW * experts;
    const int total = group_offsets(experts, s_off, s_tmp, [&](int e) { return warp_prefix(s_cnt, experts, kW, e); });
    for (int e = threadIdx.x; e <= experts; e += blockDim.x) offsets[e] = s_off[e];
    for (int64_t i = i0; i < i1; i += 32) {
      const int e = ids[i];
      if (e >= 0) {
        const int p = position[i] + cnt[e] + s_off[e];
        position[i] = p;
        order[p] = static_cast<int32_t>(i);
      }
      if (i >= total) order[i] = -1;
    }
  }
}

// The same for given ids: equal ids among 32 consecutive slots are ranked by a warp match.  Bound by the latency of
// its turns: 4 us for 777 ids, one block.
template <bool ONE>
__global__ void __launch_bounds__((ONE ? kWarpsOne : kWarps) * 32)
    k_count_ids(const int32_t* __restrict__ ids, int64_t slots, int per_warp, int groups, int32_t* __restrict__ position,
                int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ order, uint32_t* err) {
  constexpr int kW = ONE ? kWarpsOne : kWarps;
  extern __shared__ int s_cnt[];  // kW x groups, then (ONE) groups + 1 offsets
  __shared__ int s_tmp[33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_go();
  for (int i = threadIdx.x; i < kW * groups; i += blockDim.x) s_cnt[i] = 0;
  __syncthreads();
  int* cnt = s_cnt + warp * groups;
  const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * kW + warp) * per_warp;
  const int64_t i1 = min(slots, i0 + per_warp);
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
  if (!ONE) {
    for (int e = threadIdx.x; e < groups; e += blockDim.x)
      counts[static_cast<int64_t>(e) * gridDim.x + blockIdx.x] = warp_prefix(s_cnt, groups, kW, e);
    __syncthreads();
    for (int64_t i = i0 + lane; i < i1; i += 32)
      if (position[i] >= 0) position[i] += cnt[ids[i]];
  } else {
    int* s_off = s_cnt + kW * groups;
    const int total = group_offsets(groups, s_off, s_tmp, [&](int e) { return warp_prefix(s_cnt, groups, kW, e); });
    for (int e = threadIdx.x; e <= groups; e += blockDim.x) offsets[e] = s_off[e];
    for (int64_t i = i0 + lane; i < i1; i += 32) {
      if (position[i] >= 0) {
        const int e = ids[i], p = position[i] + cnt[e] + s_off[e];
        position[i] = p;
        order[p] = static_cast<int32_t>(i);
      }
      if (i >= total) order[i] = -1;
    }
  }
}

// counts[e * blocks + b] -> the slots of group e in the blocks before b; total[e] = all of them.
// One block per group, consecutive threads on consecutive blocks' counts: 4 us for 512 blocks x 64 groups
// (a warp per group over counts laid out by block: 25 us at 1024 blocks).
__global__ void __launch_bounds__(256) k_block_offsets(int32_t* __restrict__ counts, int64_t blocks,
                                                       int32_t* __restrict__ total) {
  __shared__ int s_tmp[33];
  int32_t* c = counts + blockIdx.x * blocks;
  pdl_wait();
  pdl_go();
  int run = 0;
  for (int64_t b0 = 0; b0 < blocks; b0 += blockDim.x) {
    const int64_t b = b0 + threadIdx.x;
    const int n = b < blocks ? c[b] : 0;
    int sum;
    const int incl = block_incl_scan(n, s_tmp, &sum);
    if (b < blocks) c[b] = run + incl - n;
    run += sum;
  }
  if (threadIdx.x == 0) total[blockIdx.x] = run;
}

// position: rank in the block -> position; order: its inverse; offsets.  per_block consecutive
// slots belong to one block of the counting kernel, and to one block here.  8 us for 393216 slots: scattered
// 4-byte stores.
__global__ void __launch_bounds__(kWarps * 32) k_group_scatter(const int32_t* __restrict__ ids, int64_t slots,
                                                               int64_t per_block, int groups,
                                                               const int32_t* __restrict__ counts,
                                                               const int32_t* __restrict__ total,
                                                               int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                                                               int32_t* __restrict__ position) {
  extern __shared__ int s_off[];  // groups + 1, then the block's base of each group
  __shared__ int s_tmp[33];
  pdl_wait();
  pdl_go();
  int* s_base = s_off + groups + 1;
  for (int e = threadIdx.x; e < groups; e += blockDim.x)
    s_base[e] = counts[static_cast<int64_t>(e) * gridDim.x + blockIdx.x];
  const int run = group_offsets(groups, s_off, s_tmp, [&](int e) { return total[e]; });
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= groups; e += blockDim.x) offsets[e] = s_off[e];
  const int64_t i1 = min(slots, (static_cast<int64_t>(blockIdx.x) + 1) * per_block);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x; i < i1; i += blockDim.x) {
    const int r = position[i];
    if (r >= 0) {
      const int e = ids[i];
      const int p = s_off[e] + s_base[e] + r;
      position[i] = p;
      order[p] = static_cast<int32_t>(i);
    }
    if (i >= run) order[i] = -1;  // positions behind the last group
  }
}

// Gradient of the logits; the row's scores are computed again.  A token's chosen gradients meet its row
// through shared memory.  Bound by instructions per row, like the choice: 14 us for 65536 x 64 in bf16, 17 MB
// at 1.2 TB/s, half the issue slots.
template <typename T, int L, int V>
__global__ void __launch_bounds__(kWarps * 32) k_route_backward(const T* __restrict__ logits, int64_t stride,
                                                                int64_t tokens, int experts, int pieces,
                                                                const __grid_constant__ spgemm_route_rule r,
                                                                const int32_t* __restrict__ ids,
                                                                const float* __restrict__ grad_w, T* __restrict__ out,
                                                                int64_t out_stride, int out_pieces) {
  constexpr int kPer = 32 / L;
  __shared__ float s_row[kWarps][kPer][L * V];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int me = lane & (L - 1), sub = lane / L, e0 = me * V;
  float* full = s_row[warp][sub];  // gradients of the scores of the whole row
  pdl_wait();
  pdl_go();
#pragma unroll
  for (int v = 0; v < V; ++v) full[e0 + v] = 0.0f;
  __syncwarp();
  for (int64_t tw = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kPer; tw < tokens;
       tw += static_cast<int64_t>(gridDim.x) * kWarps * kPer) {
    const int64_t t = tw + sub;
    const bool there = t < tokens;
    float l[V], s[V], d[V];
    load_row<T, L, V>(there ? logits + t * stride : nullptr, experts, pieces, l);
    const float f = row_scores<L, V>(r.score, l, s);
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] *= f;
    uint32_t chosen = 0;
    for (int j = me; there && j < r.top_k; j += L) {
      const int e = ids[t * r.top_k + j];
      if (e >= 0 && e < experts) full[e] = grad_w[t * r.top_k + j] * r.scale;
    }
    // which experts were chosen: a mark per expert in the row's own lanes
    __syncwarp();
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = full[e0 + v];
    // d becomes s times the gradient of the scores.  w = s / sum: s ds = w (dw - sum of dw w), over the chosen ones,
    // formed without ds itself, which overflows where the scores are small.
    if (r.renormalise) {
      float sum = 0.0f, mean = 0.0f;
      for (int j = 0; j < r.top_k; ++j) {
        const int e = there ? ids[t * r.top_k + j] : -1;
        if (e >= e0 && e < e0 + V && e < experts) chosen |= 1u << (e - e0);
      }
#pragma unroll
      for (int v = 0; v < V; ++v)
        if ((chosen >> v) & 1u) sum += s[v];
      sum = lanes_sum<L>(sum);
      // each weight by division, so that a single choice (weight exactly 1) has the gradient 0 exactly
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (((chosen >> v) & 1u) && sum > 0.0f) mean += d[v] * (s[v] / sum);
      mean = lanes_sum<L>(mean);
#pragma unroll
      for (int v = 0; v < V; ++v) d[v] = ((chosen >> v) & 1u) && sum > 0.0f ? s[v] / sum * (d[v] - mean) : 0.0f;
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) d[v] *= s[v];
    }
    float dot = 0.0f;
    if (r.score == SPGEMM_SCORE_SOFTMAX) {
#pragma unroll
      for (int v = 0; v < V; ++v) dot += d[v];
      dot = lanes_sum<L>(dot);
    }
    Piece<T, V> o;
#pragma unroll
    for (int v = 0; v < V; ++v)
      o.v[v] = from_f32<T>(r.score == SPGEMM_SCORE_SOFTMAX ? d[v] - s[v] * dot : d[v] * (1.0f - s[v]));
    if (there) {
      if (out_pieces && e0 + V <= experts) {
        *reinterpret_cast<Piece<T, V>*>(out + t * out_stride + e0) = o;
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (e0 + v < experts) out[t * out_stride + e0 + v] = o.v[v];
      }
    }
    __syncwarp();
#pragma unroll
    for (int v = 0; v < V; ++v) full[e0 + v] = 0.0f;
    __syncwarp();
  }
}

namespace {

template <int L_, int V_>
struct Width {
  static constexpr int L = L_, V = V_;
};

// f(Width) for the fewest lanes, then the fewest registers, that hold a row
template <typename F>
void for_width(int experts, F f) {
  if (experts <= 64) f(Width<8, 8>());
  else if (experts <= 128) f(Width<16, 8>());
  else if (experts <= 256) f(Width<32, 8>());
  else if (experts <= 512) f(Width<32, 16>());
  else f(Width<32, 32>());
}
int tokens_per_step(int experts) { return experts <= 64 ? 4 : experts <= 128 ? 2 : 1; }

// whether rows may be read in pieces of V elements (at most 16 bytes each)
template <typename T>
bool in_pieces(const spgemm_dense& d) {
  return reinterpret_cast<uintptr_t>(d.data) % 16 == 0 && (d.stride * static_cast<int64_t>(sizeof(T))) % 16 == 0;
}

struct Shape {
  bool one;
  int steps;
  int64_t blocks;
};

// One block while its warps have one step each: 64 experts, 64 tokens 7.2 us against 9.2 with three launches, 128
// tokens 10.5 against 9.6, 512 (four steps) 30 against 9.2; 256 experts, 32 tokens 8.3 against 8.2, 64 tokens 13 against
// 8.6.  Else up to kSteps steps per warp once there are two blocks per SM: 65536 x 64 40 us with one step, 36 with two,
// 39 with four; 16384 x 256 35, 29 and 30.
Shape route_shape(int64_t tokens, int experts) {
  const int64_t step = tokens_per_step(experts);
  const int64_t one = ceil_div(tokens, kWarpsOne * step);
  if (one <= 1 && experts <= kOneExperts) return {true, 1, 1};
  const int64_t steps = std::min<int64_t>(kSteps, std::max<int64_t>(1, tokens / (kWarps * step * 304)));
  return {false, static_cast<int>(steps), ceil_div(tokens, kWarps * step * steps)};
}

// One block while its warps have as many slots as those of many blocks: 1024 slots 6.2 us against 9.2 with three
// launches, 4096 slots 10.1 against 9.4, 16384 24.8 against 9.4.
Shape group_shape(int64_t slots, int groups) {
  if (slots <= kWarpsOne * kSlotsPerWarp && groups <= kOneExperts)
    return {true, static_cast<int>(std::max<int64_t>(32, ceil_div(slots, kWarpsOne * 32) * 32)), 1};
  return {false, kSlotsPerWarp, ceil_div(slots, kWarps * kSlotsPerWarp)};
}

int64_t scratch_bytes(const Shape& s, int64_t groups) { return s.one ? 0 : 4 * (s.blocks * groups + groups); }

void transpose(const int32_t* ids, int64_t slots, int64_t per_block, int64_t blocks, int groups, int32_t* counts,
               int32_t* offsets, int32_t* order, int32_t* position, cudaStream_t s) {
  int32_t* total = counts + blocks * groups;
  launch_next(k_block_offsets, static_cast<unsigned>(groups), 256, 0, s, counts, blocks, total);
  launch_next(k_group_scatter, static_cast<unsigned>(blocks), kWarps * 32, sizeof(int) * (2 * groups + 1), s, ids, slots,
              per_block, groups, static_cast<const int32_t*>(counts), static_cast<const int32_t*>(total), offsets, order,
              position);
}

}  // namespace

int64_t route_scratch_bytes(int64_t tokens, int32_t experts) { return scratch_bytes(route_shape(tokens, experts), experts); }
int64_t group_scratch_bytes(int64_t slots, int32_t groups) { return scratch_bytes(group_shape(slots, groups), groups); }

void launch_route(const spgemm_dense& logits, const spgemm_route_rule& rule, const float* bias, const RouteOut& out,
                  void* scratch, cudaStream_t s) {
  const int64_t tokens = logits.rows;
  const int experts = static_cast<int>(logits.cols);
  int32_t* counts = static_cast<int32_t*>(scratch);
  const Shape shape = route_shape(tokens, experts);
  const int step = tokens_per_step(experts);
  if (tokens == 0) {
    cudaMemsetAsync(out.offsets, 0, sizeof(int32_t) * (experts + 1), s);
    return;
  }
  for_dtype(logits.dtype, [&](auto type) {
    for_width(experts, [&](auto w) {
      using T = decltype(type);
      using W = decltype(w);
      auto go = [&](auto kern, int warps, size_t smem) {
        launch_next(kern, static_cast<unsigned>(shape.blocks), warps * 32, smem, s, static_cast<const T*>(logits.data),
                    logits.stride, tokens, experts, in_pieces<T>(logits) ? 1 : 0, shape.steps, rule, bias, out.ids,
                    out.weights, out.position, counts, out.offsets, out.order);
      };
      if constexpr (W::V == 8) {
        if (shape.one) {
          go(k_route<T, W::L, W::V, true>, kWarpsOne, sizeof(int) * (kWarpsOne * experts + experts + 1));
          return;
        }
      }
      go(k_route<T, W::L, W::V, false>, kWarps, sizeof(int) * kWarps * experts);
    });
  });
  if (!shape.one)
    transpose(out.ids, tokens * rule.top_k, static_cast<int64_t>(kWarps) * shape.steps * step * rule.top_k, shape.blocks,
              experts, counts, out.offsets, out.order, out.position, s);
}

void launch_group_rows(const int32_t* ids, int64_t slots, int32_t groups, int32_t* offsets, int32_t* order,
                       int32_t* position, void* scratch, cudaStream_t s) {
  int32_t* counts = static_cast<int32_t*>(scratch);
  const Shape shape = group_shape(slots, groups);
  if (shape.one) {
    launch_next(k_count_ids<true>, 1u, kWarpsOne * 32, sizeof(int) * (kWarpsOne * groups + groups + 1), s, ids, slots,
                shape.steps, static_cast<int>(groups), position, counts, offsets, order, grouped_err());
    return;
  }
  if (shape.blocks == 0) {
    cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (groups + 1), s);
    return;
  }
  launch_next(k_count_ids<false>, static_cast<unsigned>(shape.blocks), kWarps * 32, sizeof(int) * kWarps * groups, s, ids,
              slots, shape.steps, static_cast<int>(groups), position, counts, offsets, order, grouped_err());
  transpose(ids, slots, static_cast<int64_t>(kWarps) * kSlotsPerWarp, shape.blocks, groups, counts, offsets, order,
            position, s);
}

void launch_route_backward(const spgemm_dense& logits, const spgemm_route_rule& rule, const int32_t* ids,
                           const float* grad_w, const spgemm_dense& out, cudaStream_t s) {
  const int64_t tokens = logits.rows;
  const int experts = static_cast<int>(logits.cols);
  if (tokens == 0) return;
  const int64_t blocks = std::min<int64_t>(ceil_div(tokens, kWarps * tokens_per_step(experts)), 1 << 20);
  for_dtype(logits.dtype, [&](auto type) {
    for_width(experts, [&](auto w) {
      using T = decltype(type);
      using W = decltype(w);
      launch_next(k_route_backward<T, W::L, W::V>, static_cast<unsigned>(blocks), kWarps * 32, 0, s,
                  static_cast<const T*>(logits.data), logits.stride, tokens, experts, in_pieces<T>(logits) ? 1 : 0, rule,
                  ids, grad_w, static_cast<T*>(out.data), out.stride, in_pieces<T>(out) ? 1 : 0);
    });
  });
}

}  // namespace sg
