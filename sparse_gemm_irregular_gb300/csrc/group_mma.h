// Launchers of the tensor-core grouped products (k_group_mma.cu).
#pragma once

#include "groups.h"

namespace sg {

enum MmaMode { kMmaForward = 0, kMmaGated = 1, kMmaDx = 2, kMmaDw = 3, kMmaAdapted = 4 };

struct MmaArgs {
  const int32_t* offsets;  // NULL: one group of all rows
  const int32_t* order;
  int slots, groups, top_k;
  int rows;                // rows of the gathered matrix: the index that reads as zeros
  int gather, scatter;
  int early;               // the kernel before makes only the rows of B (or v): start without waiting for it
  int runs;                // gathered rows often follow one another
  int bf16;
  int m, n, depth;         // M side, N side (Dw only), contracted length
  int tile_n, box_rows;
  int stages, stage_bytes, sub_bytes;
  void* out;
  int64_t out_stride, out_group;
  int out_type;
  const float* scale;      // per group (scatter)
  const int32_t* ids;      // Adapted: the adapter of each row
  int adapters, rank;
  const void *x, *w, *v, *b;  // Adapted: the operands again, for sums that came out NaN or infinite
  int64_t x_stride, w_stride, v_stride, b_stride, b_group;
  int split;               // blocks that share a tile's contracted range
  uint32_t* unsure;        // Forward, 16-bit rows out: where the marks go (k_group_settle.cu), or NULL
  float near;              // sums closer than this times the largest beside them to a rounding boundary are marked
  uint32_t* err;
  uint32_t polls;          // of every wait
  int hold;                // tests: withhold an announcement
};

int sm_count();

// see spgemm_grouped_debug
void mma_debug(int32_t hold, int32_t polls);
// see spgemm_grouped_force
void mma_force(int32_t width, int32_t pair, int32_t split);

// whether the copy engine can fetch rows of this matrix: 16-bit, 16-byte aligned rows
bool mma_takes(const spgemm_dense& m);
bool mma_takes(const spgemm_weights& w);

// whether so few rows per group are expected that gathering copies keep up with the weights
bool mma_gathers(const spgemm_grouping& g);

// The same contracts as the launch_plain_* functions; false: the launch failed (cudaGetLastError
// or the encoding of a copy descriptor).
// early: x is made by the kernel launched just before on the stream, which was itself launched by launch_next or
// by these functions and makes nothing else that is read here.  unsure: mma_marks_bytes() of scratch for the marks
// that launch_settle reads, or NULL.
bool launch_mma_forward(const spgemm_grouping& g, const spgemm_dense& x, bool gather, const spgemm_weights& w,
                        bool gated, const spgemm_dense& y, uint32_t* unsure, bool early, cudaStream_t s);

// Rows of the N-side tiles that launch_mma_forward takes (not gated), about how many there are, and the bytes of
// its marks: a word per 32 rows of a tile and column of y.
int mma_forward_tile(const spgemm_grouping& g, const spgemm_dense& x, bool gather, int64_t cols);
int64_t mma_likely_tiles(const spgemm_grouping& g, int tile_n);
int64_t mma_marks_bytes(const spgemm_grouping& g, int tile_n, int64_t cols);
// Sums the marked elements of y again in index order (k_group_settle.cu); arguments as of launch_mma_forward.
bool launch_settle(const spgemm_grouping& g, const spgemm_dense& x, bool gather, const spgemm_weights& w,
                   const spgemm_dense& y, const uint32_t* unsure, int tile_n, cudaStream_t s);
bool launch_mma_dx(const spgemm_grouping& g, const spgemm_dense& dy, const spgemm_weights& w, float* dx,
                   cudaStream_t s);
// x with one row per position here
bool launch_mma_dw(const spgemm_grouping& g, const spgemm_dense& dy, const spgemm_dense& x, const spgemm_weights& dw,
                   cudaStream_t s);
// v[t, :] = scale[i] * x[t] * a[i]^T, rounded to x's type, for the rows of every adapter i
bool launch_mma_shrink(const spgemm_grouping& g, const spgemm_dense& x, const spgemm_weights& a, const float* scale,
                       const spgemm_dense& v, cudaStream_t s);
// y[t, :] = x[t] * w^T + v[t] * b[ids[t]]^T; v is made by the launch_mma_shrink just before
bool launch_mma_adapted(const spgemm_dense& x, const spgemm_dense& w, const spgemm_weights& b, const int32_t* ids,
                        const spgemm_dense& v, const spgemm_dense& y, cudaStream_t s);

}  // namespace sg
