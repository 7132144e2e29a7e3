// C entry points of the grouped-product operators: argument checks, scratch from the library's
// stream-ordered pool, and the choice between the tensor-core and the CUDA-core kernels.
#include <algorithm>
#include <atomic>
#include <initializer_list>

#include "group_mma.h"

namespace sg {

cudaMemPool_t device_pool(int dev);

static __device__ uint32_t g_grouped_err;

uint32_t* grouped_err() {
  static std::atomic<uint32_t*> at[64];  // per device: the symbol's address does not change
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  uint32_t* p = at[dev].load(std::memory_order_relaxed);
  if (!p) {
    void* v = nullptr;
    if (cudaGetSymbolAddress(&v, g_grouped_err) != cudaSuccess) cudaGetLastError();
    p = static_cast<uint32_t*>(v);
    at[dev].store(p, std::memory_order_relaxed);
  }
  return p;
}

// Reads and clears the word in one step: what another stream sets meanwhile is in this answer or in the next.
static __global__ void k_take_error(uint32_t* word, uint32_t* out) { *out = atomicExch(word, 0u); }

namespace {

constexpr int64_t kMaxSlots = (int64_t(1) << 31) - (1 << 20);  // positions and tile ends stay 32-bit

// Scratch of one call: one allocation of all its parts, returned to the pool in stream order when the
// call ends.  Parts of no bytes are null.
class Scratch {
 public:
  Scratch(cudaStream_t s, std::initializer_list<int64_t> parts) : s_(s) {
    int64_t all = 0;
    for (const int64_t b : parts) {
      at_[n_] = b ? all : -1;
      all += (b + 255) / 256 * 256;
      ++n_;
    }
    if (!all) return;
    int dev = 0;
    cudaGetDevice(&dev);
    void* p = nullptr;
    if (cudaMallocFromPoolAsync(&p, static_cast<size_t>(all), device_pool(dev), s_) != cudaSuccess) {
      cudaGetLastError();
      set_last_error("scratch allocation failed");
      ok_ = false;
      return;
    }
    base_ = static_cast<char*>(p);
  }
  ~Scratch() {
    if (base_) cudaFreeAsync(base_, s_);
  }
  Scratch(const Scratch&) = delete;
  Scratch& operator=(const Scratch&) = delete;
  template <typename T = void>
  T* part(int i) const {
    return base_ && at_[i] >= 0 ? reinterpret_cast<T*>(base_ + at_[i]) : nullptr;
  }
  bool ok() const { return ok_; }

 private:
  cudaStream_t s_;
  char* base_ = nullptr;
  int64_t at_[8];
  int n_ = 0;
  bool ok_ = true;
};

int bad(const char* what) {
  set_last_error(what);
  return SPGEMM_ERR_INVALID_ARG;
}

int launch_failed(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return check_cuda(e, what);
  set_last_error(std::string(what) + ": a copy descriptor could not be encoded");
  return SPGEMM_ERR_CUDA;
}

bool dense_ok(const spgemm_dense* d) {
  return d && d->rows >= 0 && d->cols >= 0 && d->stride >= d->cols && d->dtype >= 0 && d->dtype <= 2 &&
         (d->rows * d->cols == 0 || d->data);
}
bool weights_ok(const spgemm_weights* w) {
  return w && w->groups >= 1 && w->rows >= 1 && w->cols >= 1 && w->row_stride >= w->cols && w->group_stride >= 0 &&
         w->dtype >= 0 && w->dtype <= 2 && w->data;
}

int check_grouping(const spgemm_grouping* g, int64_t tokens) {
  if (!g || g->slots < 0 || g->top_k < 1 || g->top_k > kMaxTopK || g->groups < 1 || g->groups > kMaxGroups ||
      !g->offsets || (g->slots > 0 && (!g->order || !g->position)))
    return bad("grouping: null array, or sizes out of range");
  if (g->slots > kMaxSlots) {
    set_last_error("too many slots");
    return SPGEMM_ERR_OVERFLOW;
  }
  if (tokens >= 0 && g->slots != tokens * g->top_k) return bad("grouping: slots differ from rows * top_k");
  return SPGEMM_OK;
}

int check_rule(const spgemm_dense* logits, const spgemm_route_rule* r) {
  if (!dense_ok(logits) || !r) return bad("route: null or malformed logits or rule");
  const int64_t e = logits->cols;
  if (e < 1 || e > kMaxGroups) return bad("route: 1 to 1024 experts");
  if (r->top_k < 1 || r->top_k > kMaxTopK || r->top_k > e) return bad("route: top_k out of range");
  if (r->score < 0 || r->score > 1 || r->group_score < 0 || r->group_score > 1) return bad("route: unknown score");
  if (r->groups < 1 || r->groups > 32 || e % r->groups || r->groups_kept < 1 || r->groups_kept > r->groups)
    return bad("route: expert groups out of range");
  if (!(r->scale - r->scale == 0.0f)) return bad("route: scale is not finite");
  if (logits->rows > kMaxSlots / r->top_k) {
    set_last_error("route: too many slots");
    return SPGEMM_ERR_OVERFLOW;
  }
  return SPGEMM_OK;
}

spgemm_dense dense(void* data, int64_t rows, int64_t cols, int32_t dtype) {
  return spgemm_dense{data, rows, cols, cols, dtype, 0};
}

// x laid out in group order takes this many bytes; none where its rows are gathered or in order already
int64_t spread_bytes(const spgemm_grouping& g, const spgemm_dense& x) { return 2 * g.slots * (ceil_div(x.cols, 8) * 8); }
// lays x out in group order at `to`, its rows padded to 16 bytes
spgemm_dense spread(const spgemm_grouping& g, const spgemm_dense& x, void* to, cudaStream_t s) {
  const spgemm_dense rows{to, g.slots, x.cols, ceil_div(x.cols, 8) * 8, x.dtype, 0};
  launch_spread_rows(g, x, rows, s);
  return rows;
}
}  // namespace
}  // namespace sg

using namespace sg;

#define SG_TRY(expr)                 \
  do {                               \
    const int sg_rc = (expr);        \
    if (sg_rc != SPGEMM_OK) return sg_rc; \
  } while (0)

extern "C" {

int spgemm_route(const spgemm_dense* logits, const spgemm_route_rule* rule, const float* bias, int32_t* ids,
                 float* weights, int32_t* offsets, int32_t* order, int32_t* position, void* stream) {
  set_last_error("");
  SG_TRY(check_rule(logits, rule));
  if (!offsets || (logits->rows > 0 && (!ids || !weights || !order || !position)))
    return bad("route: null output");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Scratch scratch(st, {route_scratch_bytes(logits->rows, static_cast<int32_t>(logits->cols))});
  if (!scratch.ok()) return SPGEMM_ERR_OUT_OF_MEMORY;
  launch_route(*logits, *rule, bias, RouteOut{ids, weights, offsets, order, position}, scratch.part(0), st);
  return check_cuda(cudaGetLastError(), "route");
}

int spgemm_route_backward(const spgemm_dense* logits, const spgemm_route_rule* rule, const int32_t* ids,
                          const float* grad_weights, const spgemm_dense* grad_logits, void* stream) {
  set_last_error("");
  SG_TRY(check_rule(logits, rule));
  if (!dense_ok(grad_logits) || grad_logits->rows != logits->rows || grad_logits->cols != logits->cols ||
      grad_logits->dtype != logits->dtype)
    return bad("route backward: the gradient's shape or type differs from the logits'");
  if (logits->rows > 0 && (!ids || !grad_weights)) return bad("route backward: null input");
  launch_route_backward(*logits, *rule, ids, grad_weights, *grad_logits, static_cast<cudaStream_t>(stream));
  return check_cuda(cudaGetLastError(), "route backward");
}

int spgemm_group_rows(const int32_t* ids, int64_t slots, int32_t groups, int32_t* offsets, int32_t* order,
                      int32_t* position, void* stream) {
  set_last_error("");
  if (slots < 0 || groups < 1 || groups > kMaxGroups || !offsets || (slots > 0 && (!ids || !order || !position)))
    return bad("group rows: null array, or sizes out of range");
  if (slots > kMaxSlots) {
    set_last_error("group rows: too many slots");
    return SPGEMM_ERR_OVERFLOW;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Scratch scratch(st, {group_scratch_bytes(slots, groups)});
  if (!scratch.ok()) return SPGEMM_ERR_OUT_OF_MEMORY;
  launch_group_rows(ids, slots, groups, offsets, order, position, scratch.part(0), st);
  return check_cuda(cudaGetLastError(), "group rows");
}

int spgemm_grouped_product(const spgemm_grouping* g, const spgemm_dense* x, int32_t x_grouped, const spgemm_weights* w,
                           const spgemm_dense* y, void* stream) {
  set_last_error("");
  if (!dense_ok(x) || !weights_ok(w) || !dense_ok(y)) return bad("grouped product: malformed matrix");
  SG_TRY(check_grouping(g, x_grouped ? -1 : x->rows));
  if (x_grouped && x->rows != g->slots) return bad("grouped product: x has a row per position");
  if (w->groups != g->groups || w->cols != x->cols || y->cols != w->rows || y->rows != g->slots)
    return bad("grouped product: shapes differ");
  if (w->dtype != x->dtype || (y->dtype != x->dtype && y->dtype != SPGEMM_DTYPE_F32))
    return bad("grouped product: types differ");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (mma_takes(*x) && mma_takes(*w)) {
    const bool lay = !x_grouped && !mma_gathers(*g), gather = !x_grouped && !lay, round = y->dtype != SPGEMM_DTYPE_F32;
    const int tile_n = mma_forward_tile(*g, *x, gather, y->cols);
    Scratch scratch(st, {lay ? spread_bytes(*g, *x) : 0, round ? mma_marks_bytes(*g, tile_n, y->cols) : 0});
    if (!scratch.ok()) return SPGEMM_ERR_OUT_OF_MEMORY;
    const spgemm_dense rows = lay ? spread(*g, *x, scratch.part(0), st) : *x;
    uint32_t* marks = scratch.part<uint32_t>(1);
    if (!launch_mma_forward(*g, rows, gather, *w, false, *y, marks, lay, st) ||
        (round && !launch_settle(*g, rows, gather, *w, *y, marks, tile_n, st)))
      return launch_failed("grouped product");
  } else {
    launch_plain_forward(*g, *x, !x_grouped, *w, *y, st);
  }
  return check_cuda(cudaGetLastError(), "grouped product");
}

int spgemm_grouped_product_backward(const spgemm_grouping* g, const spgemm_dense* dy, const spgemm_dense* x,
                                    const spgemm_weights* w, const spgemm_dense* dx, const spgemm_weights* dw,
                                    void* stream) {
  set_last_error("");
  if (!dense_ok(dy) || !dense_ok(x) || !weights_ok(w) || (dx && !dense_ok(dx)) || (dw && !weights_ok(dw)))
    return bad("grouped product backward: malformed matrix");
  SG_TRY(check_grouping(g, x->rows));
  if (w->groups != g->groups || w->cols != x->cols || dy->cols != w->rows || dy->rows != g->slots)
    return bad("grouped product backward: shapes differ");
  if (dx && (dx->rows != x->rows || dx->cols != x->cols)) return bad("grouped product backward: shape of dx");
  if (dw && (dw->groups != w->groups || dw->rows != w->rows || dw->cols != w->cols))
    return bad("grouped product backward: shape of dw");
  if (dw && dw->groups > 1 && dw->group_stride < (dw->rows - 1) * dw->row_stride + dw->cols)
    return bad("grouped product backward: groups of dw overlap");
  if (w->dtype != x->dtype || dy->dtype != x->dtype || (dx && dx->dtype != x->dtype) || (dw && dw->dtype != x->dtype))
    return bad("grouped product backward: types differ");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool mma = g->slots > 0 && mma_takes(*x) && mma_takes(*dy) && mma_takes(*w);
  const bool need_dx = dx && dx->rows > 0;
  Scratch scratch(st, {need_dx ? 4 * g->slots * w->cols : 0, dw && mma ? spread_bytes(*g, *x) : 0});
  if (!scratch.ok()) return SPGEMM_ERR_OUT_OF_MEMORY;
  if (need_dx) {
    // one 32-bit row per position, summed per token afterwards: the sum is rounded once
    float* r = scratch.part<float>(0);
    if (!mma) launch_plain_dx(*g, *dy, *w, r, st);
    else if (!launch_mma_dx(*g, *dy, *w, r, st)) return launch_failed("grouped product backward");
    launch_combine(*g, nullptr, dense(r, g->slots, w->cols, SPGEMM_DTYPE_F32), *dx, st);
  }
  if (dw && !mma) launch_plain_dw(*g, *dy, *x, *dw, st);
  else if (dw && !launch_mma_dw(*g, *dy, spread(*g, *x, scratch.part(1), st), *dw, st))
    return launch_failed("grouped product backward");
  return check_cuda(cudaGetLastError(), "grouped product backward");
}

int spgemm_combine(const spgemm_grouping* g, const float* weights, const spgemm_dense* y, const spgemm_dense* out,
                   void* stream) {
  set_last_error("");
  if (!dense_ok(y) || !dense_ok(out)) return bad("combine: malformed matrix");
  SG_TRY(check_grouping(g, out->rows));
  if (y->rows != g->slots || y->cols != out->cols) return bad("combine: shapes differ");
  launch_combine(*g, weights, *y, *out, static_cast<cudaStream_t>(stream));
  return check_cuda(cudaGetLastError(), "combine");
}

int spgemm_combine_backward(const spgemm_grouping* g, const float* weights, const spgemm_dense* dout,
                            const spgemm_dense* y, const spgemm_dense* dy, float* dweights, void* stream) {
  set_last_error("");
  if (!dense_ok(dout) || !dense_ok(y) || !dense_ok(dy)) return bad("combine backward: malformed matrix");
  SG_TRY(check_grouping(g, dout->rows));
  if (g->slots > 0 && !dweights) return bad("combine backward: null dweights");
  if (y->rows != g->slots || y->cols != dout->cols || dy->rows != y->rows || dy->cols != y->cols)
    return bad("combine backward: shapes differ");
  if (dy->dtype != dout->dtype) return bad("combine backward: types of dout and dy differ");
  launch_combine_backward(*g, weights, *dout, *y, *dy, dweights, static_cast<cudaStream_t>(stream));
  return check_cuda(cudaGetLastError(), "combine backward");
}

int spgemm_experts(const spgemm_grouping* g, const float* weights, const spgemm_dense* x, const spgemm_weights* w_up,
                   const spgemm_weights* w_down, const spgemm_dense* out, void* stream) {
  set_last_error("");
  if (!dense_ok(x) || !weights_ok(w_up) || !weights_ok(w_down) || !dense_ok(out))
    return bad("experts: malformed matrix");
  SG_TRY(check_grouping(g, x->rows));
  if (g->slots > 0 && !weights) return bad("experts: null weights");
  const int64_t hidden = w_down->cols;
  if (w_up->groups != g->groups || w_down->groups != g->groups || w_up->cols != x->cols || w_up->rows != 2 * hidden ||
      out->rows != x->rows || out->cols != w_down->rows)
    return bad("experts: shapes differ");
  if (w_up->dtype != x->dtype || w_down->dtype != x->dtype || out->dtype != x->dtype)
    return bad("experts: types differ");
  if (x->rows == 0) return SPGEMM_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  spgemm_dense h = dense(nullptr, g->slots, hidden, x->dtype);
  const bool mma = mma_takes(*x) && mma_takes(*w_up) && mma_takes(h) && mma_takes(*w_down);
  const bool lay = mma && !mma_gathers(*g);
  // the down product's rows stay in 32 bits: the weighted sum is rounded once
  Scratch scratch(st, {g->slots * hidden * dtype_size(x->dtype), 4 * g->slots * out->cols,
                       !mma ? 8 * g->slots * hidden : lay ? spread_bytes(*g, *x) : 0});
  if (!scratch.ok()) return SPGEMM_ERR_OUT_OF_MEMORY;
  h.data = scratch.part(0);
  const spgemm_dense y = dense(scratch.part(1), g->slots, out->cols, SPGEMM_DTYPE_F32);
  if (mma) {
    const spgemm_dense rows = lay ? spread(*g, *x, scratch.part(2), st) : *x;
    if (!launch_mma_forward(*g, rows, !lay, *w_up, true, h, nullptr, lay, st) ||
        !launch_mma_forward(*g, h, false, *w_down, false, y, nullptr, true, st))
      return launch_failed("experts");
  } else {
    const spgemm_dense pre = dense(scratch.part(2), g->slots, 2 * hidden, SPGEMM_DTYPE_F32);
    launch_plain_forward(*g, *x, true, *w_up, pre, st);
    launch_gated(static_cast<float*>(pre.data), g->slots, hidden, h, st);
    launch_plain_forward(*g, h, false, *w_down, y, st);
  }
  launch_combine(*g, weights, y, *out, st);
  return check_cuda(cudaGetLastError(), "experts");
}

int spgemm_adapted_product(const spgemm_dense* x, const spgemm_dense* w, const spgemm_weights* a,
                           const spgemm_weights* b, const int32_t* ids, const float* scale, const spgemm_dense* y,
                           void* stream) {
  set_last_error("");
  if (!dense_ok(x) || !dense_ok(w) || !weights_ok(a) || !weights_ok(b) || !dense_ok(y))
    return bad("adapted product: malformed matrix");
  if (w->cols != x->cols || y->cols != w->rows || y->rows != x->rows || a->cols != x->cols || b->rows != y->cols ||
      a->groups != b->groups || a->rows != b->cols || w->rows < 1 || w->cols < 1)
    return bad("adapted product: shapes differ");
  if (a->groups > kMaxGroups) return bad("adapted product: more than 1024 adapters");
  if (w->dtype != x->dtype || a->dtype != x->dtype || b->dtype != x->dtype || y->dtype != x->dtype)
    return bad("adapted product: types differ");
  if (x->rows > kMaxSlots) {
    set_last_error("adapted product: too many rows");
    return SPGEMM_ERR_OVERFLOW;
  }
  if (x->rows == 0) return SPGEMM_OK;
  if (!ids) return bad("adapted product: null ids");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t t = x->rows, rank = a->rows;
  const int32_t adapters = static_cast<int32_t>(a->groups);
  // v is rounded to x's type between the two small products on the tensor cores, 32-bit otherwise
  spgemm_dense v{nullptr, t, rank, ceil_div(rank, 8) * 8, x->dtype, 0};
  const bool mma = mma_takes(*x) && mma_takes(*w) && mma_takes(*a) && mma_takes(*b) && mma_takes(v);
  if (!mma) v = dense(nullptr, t, rank, SPGEMM_DTYPE_F32);
  Scratch scratch(st, {4 * (adapters + 1), 4 * t, 4 * t, group_scratch_bytes(t, adapters), t * v.stride * dtype_size(v.dtype),
                       mma ? 0 : 4 * t * y->cols});
  if (!scratch.ok()) return SPGEMM_ERR_OUT_OF_MEMORY;
  int32_t *offsets = scratch.part<int32_t>(0), *order = scratch.part<int32_t>(1), *position = scratch.part<int32_t>(2);
  v.data = scratch.part(4);
  launch_group_rows(ids, t, adapters, offsets, order, position, scratch.part(3), st);
  const spgemm_grouping g{t, 1, adapters, offsets, order, position};
  if (mma) {
    if (!launch_mma_shrink(g, *x, *a, scale, v, st) || !launch_mma_adapted(*x, *w, *b, ids, v, *y, st))
      return launch_failed("adapted product");
  } else {
    const spgemm_dense base = dense(scratch.part(5), t, y->cols, SPGEMM_DTYPE_F32);
    launch_plain_forward(g, *x, true, *a, v, st);
    const spgemm_weights shared{w->data, 1, w->rows, w->cols, 0, w->stride, w->dtype, 0};
    launch_plain_forward(spgemm_grouping{t, 1, 1, nullptr, nullptr, nullptr}, *x, false, shared, base, st);
    launch_plain_adapter_add(g, ids, scale, static_cast<float*>(base.data), static_cast<float*>(v.data), rank, *b, *y, st);
  }
  return check_cuda(cudaGetLastError(), "adapted product");
}

int spgemm_grouped_debug(int32_t hold, int32_t polls) {
  if (polls < 0) return bad("grouped debug: negative polls");
  mma_debug(hold, polls);
  return SPGEMM_OK;
}

int spgemm_grouped_force(int32_t width, int32_t pair, int32_t split) {
  const bool two = width >= 16 && width <= 256 && (width & (width - 1)) == 0;
  if ((width && !two) || pair < 0 || pair > 1 || split < 0 || split > 8) return bad("grouped force: out of range");
  mma_force(width, pair, split);
  return SPGEMM_OK;
}

int spgemm_grouped_status(void* stream) {
  set_last_error("");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t* p = grouped_err();
  if (!p) return check_cuda(cudaErrorInvalidSymbol, "grouped status");
  uint32_t err = 0;
  {
    Scratch scratch(st, {sizeof(err)});
    if (!scratch.ok()) return SPGEMM_ERR_OUT_OF_MEMORY;
    note_launch();
    k_take_error<<<1, 1, 0, st>>>(p, scratch.part<uint32_t>(0));
    SG_TRY(check_cuda(cudaGetLastError(), "grouped status"));
    SG_TRY(check_cuda(cudaMemcpyAsync(&err, scratch.part(0), sizeof(err), cudaMemcpyDeviceToHost, st), "grouped status"));
    SG_TRY(check_cuda(cudaStreamSynchronize(st), "grouped status"));
  }
  if (!err) return SPGEMM_OK;
  if (err & kErrTimeout) set_last_error("a wait expired (sites " + std::to_string(err >> 8) + ")");
  else set_last_error("an id is outside its range");
  return SPGEMM_ERR_DEVICE;
}

}  // extern "C"
