// C-ABI front end of the expert-parallel exchange and products: argument
// validation, workspace layout and dispatch to the kernels.  Every check
// runs before the first HIP call, so a rejected call enqueues nothing.

#include <algorithm>
#include <cstdio>

#include "ccl_sim.h"
#include "experts.hpp"
#include "front.hpp"

namespace {

using namespace ccl;

using Shape = ccl_sim_expert_shape_t;
using Arrays = const void* const*;

constexpr size_t kMaxWidth = size_t(1) << 20;
constexpr int kMaxArrays = 8;

bool row_type(int dtype) { return dtype == CCL_SIM_FLOAT32 || dtype == CCL_SIM_BFLOAT16; }
bool any_type(int dtype) { return dtype >= CCL_SIM_INT32 && dtype <= CCL_SIM_BFLOAT16; }
bool is_product(int op) { return op == CCL_SIM_EXPERT_MATMUL || op == CCL_SIM_EXPERT_MATMUL_GRAD; }

// The shape's fields that `op` reads.
ccl_sim_result_t check_shape(int op, const Shape* s) {
  if (s == nullptr) return fail(CCL_SIM_INVALID_ARGUMENT, "shape is NULL");
  if (s->nranks < 1 || s->nranks > CCL_SIM_MAX_RANKS)
    return fail(CCL_SIM_INVALID_ARGUMENT, "nranks=%d outside [1, %d]", s->nranks, CCL_SIM_MAX_RANKS);
  const uint64_t n = uint64_t(s->nranks), limit = uint64_t(1) << 31;
  if (s->capacity >= limit || n * s->capacity >= limit)
    return fail(CCL_SIM_INVALID_ARGUMENT, "nranks (%d) x capacity (%zu) is not below 2^31", s->nranks, s->capacity);
  if (op == CCL_SIM_EXPERT_ROUTE || is_product(op)) {
    if (s->experts < 1 || s->experts > CCL_SIM_MAX_EXPERTS || s->experts % s->nranks != 0)
      return fail(CCL_SIM_INVALID_ARGUMENT, "experts=%d is not a multiple of nranks (%d) in [1, %d]", s->experts,
                  s->nranks, CCL_SIM_MAX_EXPERTS);
  }
  if (!is_product(op)) {
    if (s->topk < 1 || s->topk > CCL_SIM_MAX_TOPK)
      return fail(CCL_SIM_INVALID_ARGUMENT, "topk=%d outside [1, %d]", s->topk, CCL_SIM_MAX_TOPK);
    if (s->tokens >= limit || n * uint64_t(s->topk) * s->tokens >= limit)
      return fail(CCL_SIM_INVALID_ARGUMENT, "nranks (%d) x tokens (%zu) x topk (%d) is not below 2^31", s->nranks,
                  s->tokens, s->topk);
  }
  if (op != CCL_SIM_EXPERT_ROUTE && s->hidden > kMaxWidth)
    return fail(CCL_SIM_INVALID_ARGUMENT, "hidden=%zu is above %zu", s->hidden, kMaxWidth);
  if (is_product(op)) {
    if (s->features > kMaxWidth)
      return fail(CCL_SIM_INVALID_ARGUMENT, "features=%zu is above %zu", s->features, kMaxWidth);
    if (s->hidden == 0) return fail(CCL_SIM_INVALID_ARGUMENT, "a product over hidden=0 elements");
    // a launch holds fewer than 2^32 threads: 256 to 64 rows or more and 128
    // columns or more (the pass over the activation's gradient), 256 to 64
    // columns of an expert (few rows).  The tile kernel's workgroups take
    // turns; its tiles are counted in 32 bits.
    const uint64_t per_rank = uint64_t(s->experts / s->nranks), f = s->features / 128 + 1, h = s->hidden / 128 + 1;
    const uint64_t tiles = std::max({n * (s->capacity / 64 + per_rank) * std::max(f, h), uint64_t(s->experts) * f * h,
                                     uint64_t(s->experts) * (s->features / 64 + 1)});
    if (tiles >= (uint64_t(1) << 24))
      return fail(CCL_SIM_INVALID_ARGUMENT, "a product of %llu tiles does not fit one launch",
                  static_cast<unsigned long long>(tiles));
  } else if (op != CCL_SIM_EXPERT_ROUTE) {
    if (n * s->tokens * (s->hidden / 128 + 1) >= limit)
      return fail(CCL_SIM_INVALID_ARGUMENT, "nranks (%d) x tokens (%zu) rows of %zu elements do not fit one launch",
                  s->nranks, s->tokens, s->hidden);
  }
  return CCL_SIM_SUCCESS;
}

// Workspace layout: the pointer tables of all the arrays an op may have
// (nranks > 64), then the op's own parts.
struct Layout {
  size_t tables = 0, table_bytes = 0;
  size_t own = 0;    // where the op's own parts start
  size_t total = 0;
};

// The sizes below stay within 64 bits for every shape that check_shape lets
// through: nranks·capacity < 2^31, widths <= 2^20, elements <= 8 bytes.
Layout layout(int op, const Shape& s, int dtype) {
  Layout l;
  size_t off = 0;
  if (s.nranks > kInlineRanks) {
    l.table_bytes = round_up(size_t(s.nranks) * sizeof(void*));
    off += kMaxArrays * l.table_bytes;
  }
  l.own = off;
  if (op == CCL_SIM_EXPERT_ROUTE) {
    const RoutePlan plan = route_plan(uint64_t(s.nranks) * s.tokens * uint64_t(s.topk), s.experts);
    if (plan.in_memory) off += round_up((size_t(plan.blocks) + 1) * size_t(s.experts) * sizeof(int));
  }
  if (is_product(op)) {
    const ProductPlan plan = product_plan(dtype, uint32_t(s.nranks), uint32_t(s.experts / s.nranks),
                                          uint32_t(s.capacity), uint32_t(s.hidden), uint32_t(s.features));
    off += op == CCL_SIM_EXPERT_MATMUL ? plan.forward : plan.grads;
  }
  l.total = off;
  return l;
}

// One array argument: its pointers, the bytes of a rank's buffer, the
// alignment it needs, and how it may overlap.
struct Array {
  const char* name;
  Arrays ptrs;
  uint64_t bytes;
  size_t align;
  bool output;
  int same_as;       // an output that may be this input's buffers, else -1
  RankPtrs* to;      // where the kernels' copy goes
  bool used = true;  // the call has it: its kernels ask for its addresses, also where it has no elements

  bool touched() const { return used && bytes > 0; }
};

// The addresses of arrays without elements.
const void* const kNowhere[CCL_SIM_MAX_RANKS] = {};

struct Span {
  uintptr_t lo, hi;
  int rank, array;
};

// Outputs are pairwise disjoint, and disjoint from the inputs and the
// workspace, except for an output that is its `same_as` input's buffer of
// the same rank.  Sorts the outputs: O(N log N).
ccl_sim_result_t check_overlap(const Array* arrays, int count, int nranks, uintptr_t ws, uintptr_t ws_end) {
  Span outs[3 * CCL_SIM_MAX_RANKS];
  int n = 0;
  for (int i = 0; i < count; ++i)
    if (arrays[i].output && arrays[i].touched())
      for (int r = 0; r < nranks; ++r) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(arrays[i].ptrs[r]);
        outs[n++] = Span{p, p + arrays[i].bytes, r, i};
      }
  std::sort(outs, outs + n, [](const Span& a, const Span& b) { return a.lo < b.lo; });
  for (int i = 1; i < n; ++i)
    if (outs[i - 1].hi > outs[i].lo)
      return fail(CCL_SIM_INVALID_ARGUMENT, "outputs %s[%d] and %s[%d] overlap", arrays[outs[i - 1].array].name,
                  outs[i - 1].rank, arrays[outs[i].array].name, outs[i].rank);
  auto first_past = [&](uintptr_t lo) {
    return std::upper_bound(outs, outs + n, lo, [](uintptr_t v, const Span& s) { return v < s.hi; });
  };
  for (int i = 0; i < count; ++i) {
    if (!arrays[i].touched()) continue;
    for (int r = 0; r < nranks; ++r) {
      const uintptr_t lo = reinterpret_cast<uintptr_t>(arrays[i].ptrs[r]), hi = lo + arrays[i].bytes;
      if (ws < hi && lo < ws_end)
        return fail(CCL_SIM_INVALID_ARGUMENT, "the workspace overlaps %s[%d]", arrays[i].name, r);
      if (arrays[i].output) continue;
      for (const Span* o = first_past(lo); o < outs + n && o->lo < hi; ++o)
        if (!(arrays[o->array].same_as == i && o->rank == r && o->lo == lo))
          return fail(CCL_SIM_INVALID_ARGUMENT, "%s[%d] overlaps the output %s[%d]", arrays[i].name, r,
                      arrays[o->array].name, o->rank);
    }
  }
  return CCL_SIM_SUCCESS;
}

// Checks the arrays and the workspace, then hands the pointers over: in the
// call itself, or by tables in the workspace.
ccl_sim_result_t bind(const Array* arrays, int count, int nranks, const Layout& lay, void* workspace,
                      size_t workspace_bytes, hipStream_t stream) {
  for (int i = 0; i < count; ++i) {
    if (!arrays[i].touched()) continue;
    const ccl_sim_result_t rc = check_ptrs(arrays[i].ptrs, nranks, arrays[i].name, arrays[i].align);
    if (rc != CCL_SIM_SUCCESS) return rc;
  }
  const uintptr_t ws = reinterpret_cast<uintptr_t>(workspace);
  if (lay.total > 0) {
    if (workspace == nullptr || workspace_bytes < lay.total)
      return fail(CCL_SIM_INSUFFICIENT_WORKSPACE, "workspace of %zu bytes needed, %zu given%s", lay.total,
                  workspace == nullptr ? size_t(0) : workspace_bytes, workspace == nullptr ? " (NULL)" : "");
    if (ws % kAlign != 0) return fail(CCL_SIM_INVALID_ARGUMENT, "workspace is not 256-byte aligned");
  }
  const ccl_sim_result_t rc = check_overlap(arrays, count, nranks, ws, ws + lay.total);
  if (rc != CCL_SIM_SUCCESS) return rc;
  for (int i = 0; i < count; ++i) {
    if (!arrays[i].used) continue;
    const Arrays ptrs = arrays[i].bytes > 0 ? arrays[i].ptrs : kNowhere;
    if (nranks <= kInlineRanks) {
      for (int r = 0; r < nranks; ++r) arrays[i].to->p[r] = ptrs[r];
    } else {
      const void** table = reinterpret_cast<const void**>(static_cast<char*>(workspace) + size_t(i) * lay.table_bytes);
      const hipError_t e = upload_table(table, ptrs, nranks, stream);
      if (e != hipSuccess) return fail(CCL_SIM_HIP_ERROR, "pointer table upload failed: %s", hipGetErrorString(e));
      arrays[i].to->table = reinterpret_cast<const uint64_t*>(table);
    }
  }
  if (lay.total > lay.own && debug_enabled()) {
    const hipError_t e = poison_fill(static_cast<char*>(workspace) + lay.own, lay.total - lay.own, stream);
    if (e != hipSuccess) return fail(CCL_SIM_HIP_ERROR, "scratch poison fill failed: %s", hipGetErrorString(e));
  }
  return CCL_SIM_SUCCESS;
}

bool starts16(Arrays ptrs, int nranks) {
  for (int r = 0; r < nranks; ++r)
    if (reinterpret_cast<uintptr_t>(ptrs[r]) % 16 != 0) return false;
  return true;
}

ccl_sim_result_t done(hipError_t e, const char* what, const Shape& s) {
  if (e != hipSuccess) return fail(CCL_SIM_HIP_ERROR, "kernel launch failed: %s", hipGetErrorString(e));
  if (debug_enabled())
    std::fprintf(stderr, "[ccl_sim] expert %s N=%d E=%d k=%d T=%zu C=%zu H=%zu F=%zu\n", what, s.nranks, s.experts, s.topk,
                 s.tokens, s.capacity, s.hidden, s.features);
  return CCL_SIM_SUCCESS;
}

Arrays as_in(void* const* p) { return const_cast<Arrays>(p); }

ExchangeCall exchange_call(const Shape& s, int dtype, ccl_sim_stream_t stream) {
  ExchangeCall c;
  c.dtype = dtype;
  c.nranks = s.nranks;
  c.experts = s.experts;
  c.topk = s.topk;
  c.tokens = uint32_t(s.tokens);
  c.capacity = uint32_t(s.capacity);
  c.hidden = s.hidden;
  c.stream = reinterpret_cast<hipStream_t>(stream);
  return c;
}

ProductCall product_call(const Shape& s, int dtype, int activation, ccl_sim_stream_t stream) {
  ProductCall c;
  c.dtype = dtype;
  c.activation = activation;
  c.nranks = s.nranks;
  c.per_rank = uint32_t(s.experts / s.nranks);
  c.capacity = uint32_t(s.capacity);
  c.hidden = uint32_t(s.hidden);
  c.features = uint32_t(s.features);
  c.log_plan = debug_enabled();
  c.stream = reinterpret_cast<hipStream_t>(stream);
  return c;
}

ccl_sim_result_t check_product(const Shape* s, int op, int dtype, int activation, bool has_offsets) {
  const ccl_sim_result_t rc = check_shape(op, s);
  if (rc != CCL_SIM_SUCCESS) return rc;
  if (!row_type(dtype))
    return fail(CCL_SIM_INVALID_ARGUMENT, "dtype %d: the products take float32 and bf16", dtype);
  if (activation < CCL_SIM_ACT_NONE || activation > CCL_SIM_ACT_SILU)
    return fail(CCL_SIM_INVALID_ARGUMENT, "invalid activation %d", activation);
  if (!has_offsets && s->experts != s->nranks)
    return fail(CCL_SIM_INVALID_ARGUMENT, "offsets may be NULL only with one expert per rank (experts=%d, nranks=%d)",
                s->experts, s->nranks);
  return CCL_SIM_SUCCESS;
}

}  // namespace

extern "C" {

size_t ccl_sim_expert_workspace_size(ccl_sim_expert_op_t op, const ccl_sim_expert_shape_t* shape,
                                     ccl_sim_dtype_t dtype) {
  clear_error();
  if (op < CCL_SIM_EXPERT_ROUTE || op > CCL_SIM_EXPERT_MATMUL_GRAD) {
    (void)fail(CCL_SIM_INVALID_ARGUMENT, "invalid expert operator %d", int(op));
    return SIZE_MAX;
  }
  if (check_shape(op, shape) != CCL_SIM_SUCCESS) return SIZE_MAX;
  const bool typed = op == CCL_SIM_EXPERT_ROUTE || (op == CCL_SIM_EXPERT_DISPATCH ? any_type(dtype) : row_type(dtype));
  if (!typed) {
    (void)fail(CCL_SIM_INVALID_ARGUMENT, "dtype %d is not one of the operator's", int(dtype));
    return SIZE_MAX;
  }
  return layout(op, *shape, dtype).total;
}

ccl_sim_result_t ccl_sim_expert_route(const ccl_sim_expert_shape_t* shape, const void* const* ids,
                                      ccl_sim_dtype_t id_dtype, int32_t* const* places, int32_t* const* offsets,
                                      void* workspace, size_t workspace_bytes, ccl_sim_stream_t stream) {
  clear_error();
  ccl_sim_result_t rc = check_shape(CCL_SIM_EXPERT_ROUTE, shape);
  if (rc != CCL_SIM_SUCCESS) return rc;
  if (id_dtype != CCL_SIM_INT32 && id_dtype != CCL_SIM_INT64)
    return fail(CCL_SIM_INVALID_ARGUMENT, "ids are int32 or int64 (dtype %d)", int(id_dtype));
  const Shape& s = *shape;
  const uint64_t choices = s.tokens * uint64_t(s.topk), entries = uint64_t(s.experts / s.nranks) + 1;
  ExchangeCall c = exchange_call(s, id_dtype, stream);
  const Layout lay = layout(CCL_SIM_EXPERT_ROUTE, s, id_dtype);
  const Array arrays[] = {
      {"ids", ids, choices * elem_size(id_dtype), elem_size(id_dtype), false, -1, &c.in},
      {"places", reinterpret_cast<Arrays>(places), choices * 4, 4, true, -1, &c.places},
      {"offsets", reinterpret_cast<Arrays>(offsets), entries * 4, 4, true, -1, &c.offsets},
  };
  rc = bind(arrays, 3, s.nranks, lay, workspace, workspace_bytes, c.stream);
  if (rc != CCL_SIM_SUCCESS) return rc;
  c.counts = reinterpret_cast<int*>(static_cast<char*>(workspace) + lay.own);
  return done(run_expert_route(c), "route", s);
}

ccl_sim_result_t ccl_sim_expert_dispatch(const ccl_sim_expert_shape_t* shape, const void* const* sendbufs,
                                         const int32_t* const* places, void* const* recvbufs, ccl_sim_dtype_t dtype,
                                         void* workspace, size_t workspace_bytes, ccl_sim_stream_t stream) {
  clear_error();
  ccl_sim_result_t rc = check_shape(CCL_SIM_EXPERT_DISPATCH, shape);
  if (rc != CCL_SIM_SUCCESS) return rc;
  if (!any_type(dtype)) return fail(CCL_SIM_INVALID_ARGUMENT, "invalid dtype %d", int(dtype));
  const Shape& s = *shape;
  if (s.tokens == 0 || s.hidden == 0 || s.capacity == 0) return CCL_SIM_SUCCESS;  // nothing to move
  const size_t es = elem_size(dtype);
  ExchangeCall c = exchange_call(s, dtype, stream);
  const Array arrays[] = {
      {"sendbufs", sendbufs, s.tokens * s.hidden * es, es, false, -1, &c.in},
      {"places", reinterpret_cast<Arrays>(places), s.tokens * uint64_t(s.topk) * 4, 4, false, -1, &c.places},
      {"recvbufs", as_in(recvbufs), s.capacity * s.hidden * es, es, true, -1, &c.out},
  };
  rc = bind(arrays, 3, s.nranks, layout(CCL_SIM_EXPERT_DISPATCH, s, dtype), workspace, workspace_bytes, c.stream);
  if (rc != CCL_SIM_SUCCESS) return rc;
  return done(run_expert_dispatch(c), "dispatch", s);
}

ccl_sim_result_t ccl_sim_expert_combine(const ccl_sim_expert_shape_t* shape, const void* const* sendbufs,
                                        const int32_t* const* places, const float* const* weights,
                                        const void* const* residual, void* const* recvbufs, ccl_sim_dtype_t dtype,
                                        void* workspace, size_t workspace_bytes, ccl_sim_stream_t stream) {
  clear_error();
  ccl_sim_result_t rc = check_shape(CCL_SIM_EXPERT_COMBINE, shape);
  if (rc != CCL_SIM_SUCCESS) return rc;
  if (!row_type(dtype)) return fail(CCL_SIM_INVALID_ARGUMENT, "dtype %d: combine takes float32 and bf16", int(dtype));
  const Shape& s = *shape;
  if (s.tokens == 0 || s.hidden == 0) return CCL_SIM_SUCCESS;
  const size_t es = elem_size(dtype);
  const uint64_t choices = s.tokens * uint64_t(s.topk), tokens = s.tokens * s.hidden * es;
  ExchangeCall c = exchange_call(s, dtype, stream);
  c.has_weights = weights != nullptr;
  c.has_residual = residual != nullptr;
  const Array arrays[] = {
      {"sendbufs", sendbufs, s.capacity * s.hidden * es, es, false, -1, &c.rows},
      {"places", reinterpret_cast<Arrays>(places), choices * 4, 4, false, -1, &c.places},
      {"weights", reinterpret_cast<Arrays>(weights), choices * 4, 4, false, -1, &c.weights, c.has_weights},
      {"residual", residual, tokens, es, false, -1, &c.residual, c.has_residual},
      {"recvbufs", as_in(recvbufs), tokens, es, true, 3, &c.out},
  };
  rc = bind(arrays, 5, s.nranks, layout(CCL_SIM_EXPERT_COMBINE, s, dtype), workspace, workspace_bytes, c.stream);
  if (rc != CCL_SIM_SUCCESS) return rc;
  return done(run_expert_combine(c), "combine", s);
}

ccl_sim_result_t ccl_sim_expert_combine_grad(const ccl_sim_expert_shape_t* shape, const void* const* grads,
                                             const void* const* sendbufs, const int32_t* const* places,
                                             const float* const* weights, void* const* grad_rows,
                                             float* const* grad_weights, ccl_sim_dtype_t dtype, void* workspace,
                                             size_t workspace_bytes, ccl_sim_stream_t stream) {
  clear_error();
  ccl_sim_result_t rc = check_shape(CCL_SIM_EXPERT_COMBINE_GRAD, shape);
  if (rc != CCL_SIM_SUCCESS) return rc;
  if (!row_type(dtype))
    return fail(CCL_SIM_INVALID_ARGUMENT, "dtype %d: combine's gradient takes float32 and bf16", int(dtype));
  const Shape& s = *shape;
  ExchangeCall c = exchange_call(s, dtype, stream);
  c.has_grad_rows = grad_rows != nullptr;
  c.has_grad_weights = grad_weights != nullptr;
  c.has_weights = weights != nullptr && c.has_grad_rows;
  if (s.tokens == 0 || (!c.has_grad_rows && !c.has_grad_weights)) return CCL_SIM_SUCCESS;
  const size_t es = elem_size(dtype);
  const uint64_t choices = s.tokens * uint64_t(s.topk), rows = s.capacity * s.hidden * es;
  const Array arrays[] = {
      {"grads", grads, s.tokens * s.hidden * es, es, false, -1, &c.in},
      {"sendbufs", sendbufs, rows, es, false, -1, &c.rows, c.has_grad_weights},
      {"places", reinterpret_cast<Arrays>(places), choices * 4, 4, false, -1, &c.places},
      {"weights", reinterpret_cast<Arrays>(weights), choices * 4, 4, false, -1, &c.weights, c.has_weights},
      {"grad_rows", as_in(grad_rows), rows, es, true, -1, &c.grad_rows, c.has_grad_rows},
      {"grad_weights", reinterpret_cast<Arrays>(grad_weights), choices * 4, 4, true, -1, &c.grad_weights,
       c.has_grad_weights},
  };
  rc = bind(arrays, 6, s.nranks, layout(CCL_SIM_EXPERT_COMBINE_GRAD, s, dtype), workspace, workspace_bytes, c.stream);
  if (rc != CCL_SIM_SUCCESS) return rc;
  const hipError_t e = device_cus(&c.num_cus);
  if (e != hipSuccess) return fail(CCL_SIM_HIP_ERROR, "device query failed: %s", hipGetErrorString(e));
  return done(run_expert_combine_grad(c), "combine_grad", s);
}

ccl_sim_result_t ccl_sim_expert_matmul(const ccl_sim_expert_shape_t* shape, const void* const* rows,
                                       const int32_t* const* offsets, const void* const* weights,
                                       const void* const* bias, const void* const* residual, void* const* preact,
                                       void* const* out, ccl_sim_dtype_t dtype, ccl_sim_activation_t activation,
                                       void* workspace, size_t workspace_bytes, ccl_sim_stream_t stream) {
  clear_error();
  ccl_sim_result_t rc = check_product(shape, CCL_SIM_EXPERT_MATMUL, dtype, activation, offsets != nullptr);
  if (rc != CCL_SIM_SUCCESS) return rc;
  const Shape& s = *shape;
  if (s.capacity == 0 || s.features == 0) return CCL_SIM_SUCCESS;
  const size_t es = elem_size(dtype);
  const uint64_t per_rank = uint64_t(s.experts / s.nranks), outs = s.capacity * s.features * es;
  ProductCall c = product_call(s, dtype, activation, stream);
  c.has_offsets = offsets != nullptr;
  c.has_bias = bias != nullptr;
  c.has_residual = residual != nullptr;
  c.has_preact = preact != nullptr;
  const Array arrays[] = {
      {"rows", rows, s.capacity * s.hidden * es, es, false, -1, &c.rows},
      {"offsets", reinterpret_cast<Arrays>(offsets), (per_rank + 1) * 4, 4, false, -1, &c.offsets, c.has_offsets},
      {"weights", weights, per_rank * s.features * s.hidden * es, es, false, -1, &c.weights},
      {"bias", bias, per_rank * s.features * es, es, false, -1, &c.bias, c.has_bias},
      {"residual", residual, outs, es, false, -1, &c.residual, c.has_residual},
      {"preact", as_in(preact), outs, es, true, -1, &c.preact, c.has_preact},
      {"out", as_in(out), outs, es, true, 4, &c.out},
  };
  const Layout lay = layout(CCL_SIM_EXPERT_MATMUL, s, dtype);
  rc = bind(arrays, 7, s.nranks, lay, workspace, workspace_bytes, c.stream);
  if (rc != CCL_SIM_SUCCESS) return rc;
  c.scratch = static_cast<char*>(workspace) + lay.own;
  c.rows16 = starts16(rows, s.nranks);
  c.weights16 = starts16(weights, s.nranks);
  const hipError_t e = device_cus(&c.num_cus);
  if (e != hipSuccess) return fail(CCL_SIM_HIP_ERROR, "device query failed: %s", hipGetErrorString(e));
  return done(run_expert_matmul(c), "matmul", s);
}

ccl_sim_result_t ccl_sim_expert_matmul_grad(const ccl_sim_expert_shape_t* shape, const void* const* grads,
                                            const void* const* rows, const int32_t* const* offsets,
                                            const void* const* weights, const void* const* preact,
                                            void* const* grad_rows, void* const* grad_weights,
                                            void* const* grad_bias, ccl_sim_dtype_t dtype,
                                            ccl_sim_activation_t activation, void* workspace,
                                            size_t workspace_bytes, ccl_sim_stream_t stream) {
  clear_error();
  ccl_sim_result_t rc = check_product(shape, CCL_SIM_EXPERT_MATMUL_GRAD, dtype, activation, offsets != nullptr);
  if (rc != CCL_SIM_SUCCESS) return rc;
  const Shape& s = *shape;
  ProductCall c = product_call(s, dtype, activation, stream);
  c.has_offsets = offsets != nullptr;
  c.has_preact = activation != CCL_SIM_ACT_NONE;
  c.want_rows = grad_rows != nullptr && s.capacity > 0;
  c.want_weights = grad_weights != nullptr;
  c.want_bias = grad_bias != nullptr;
  if (s.features == 0 && !c.want_rows) return CCL_SIM_SUCCESS;
  if (!c.want_rows && !c.want_weights && !c.want_bias) return CCL_SIM_SUCCESS;
  const size_t es = elem_size(dtype);
  const uint64_t per_rank = uint64_t(s.experts / s.nranks);
  const uint64_t wide = s.capacity * s.features * es, narrow = s.capacity * s.hidden * es;
  const uint64_t matrices = per_rank * s.features * s.hidden * es;
  const Array arrays[] = {
      {"grads", grads, wide, es, false, -1, &c.grads},
      {"rows", rows, narrow, es, false, -1, &c.rows, c.want_weights},
      {"offsets", reinterpret_cast<Arrays>(offsets), (per_rank + 1) * 4, 4, false, -1, &c.offsets, c.has_offsets},
      {"weights", weights, matrices, es, false, -1, &c.weights, c.want_rows},
      {"preact", preact, wide, es, false, -1, &c.preact, c.has_preact},
      {"grad_rows", as_in(grad_rows), narrow, es, true, -1, &c.grad_rows, c.want_rows},
      {"grad_weights", as_in(grad_weights), matrices, es, true, -1, &c.grad_weights, c.want_weights},
      {"grad_bias", as_in(grad_bias), per_rank * s.features * es, es, true, -1, &c.grad_bias, c.want_bias},
  };
  const Layout lay = layout(CCL_SIM_EXPERT_MATMUL_GRAD, s, dtype);
  rc = bind(arrays, 8, s.nranks, lay, workspace, workspace_bytes, c.stream);
  if (rc != CCL_SIM_SUCCESS) return rc;
  c.scratch = static_cast<char*>(workspace) + lay.own;
  // an array without elements may be NULL
  c.rows16 = c.want_weights && narrow > 0 && starts16(rows, s.nranks);
  c.weights16 = c.want_rows && matrices > 0 && starts16(weights, s.nranks);
  c.grads16 = wide > 0 && starts16(grads, s.nranks);
  const hipError_t e = device_cus(&c.num_cus);
  if (e != hipSuccess) return fail(CCL_SIM_HIP_ERROR, "device query failed: %s", hipGetErrorString(e));
  return done(run_expert_matmul_grad(c), "matmul_grad", s);
}

}  // extern "C"
