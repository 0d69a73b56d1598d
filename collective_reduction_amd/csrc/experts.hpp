// Internal interface between the expert front end (experts.cpp: checks and
// planning) and its kernels (kernels_exchange.hip, kernels_products.hip).
// Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ccl_sim.h"
#include "device.hpp"

namespace ccl {

// A validated call of the exchange (route, dispatch, combine and its
// gradient).  Arrays a call does not have hold null pointers.
struct ExchangeCall {
  int dtype = 0;   // of the rows; of the ids for route
  int nranks = 0, experts = 0, topk = 0;
  uint32_t tokens = 0, capacity = 0;
  uint64_t hidden = 0;
  bool has_rows = false, has_weights = false, has_residual = false, has_grad_rows = false, has_grad_weights = false;
  // route: ids -> places, offsets; dispatch: in -> out; combine: rows -> out;
  // combine_grad: in (the gradients), rows -> grad_rows, grad_weights
  RankPtrs in{}, rows{}, places{}, offsets{}, weights{}, residual{}, out{}, grad_rows{}, grad_weights{};
  int* counts = nullptr;  // route: [blocks][experts], then [experts] totals
  hipStream_t stream = nullptr;
  int num_cus = 0;
};

// How route splits its work: the choices one workgroup takes, the number of
// workgroups, and whether it needs counts in memory (three launches) or one
// workgroup does everything in one launch.
struct RoutePlan {
  uint32_t chunk = 0, blocks = 0;
  bool in_memory = false;  // the counts per workgroup are kept in memory
};
RoutePlan route_plan(uint64_t choices, int experts);

hipError_t run_expert_route(const ExchangeCall& c);
hipError_t run_expert_dispatch(const ExchangeCall& c);
hipError_t run_expert_combine(const ExchangeCall& c);
hipError_t run_expert_combine_grad(const ExchangeCall& c);

// A validated call of the products or of their gradients.
struct ProductCall {
  int dtype = 0, activation = 0, nranks = 0;
  uint32_t per_rank = 0;  // experts of a rank
  uint32_t capacity = 0, hidden = 0, features = 0;
  bool has_offsets = false, has_bias = false, has_residual = false, has_preact = false;
  bool want_rows = false, want_weights = false, want_bias = false;  // the gradients asked for
  RankPtrs rows{}, offsets{}, weights{}, bias{}, residual{}, preact{}, out{};
  RankPtrs grads{}, grad_rows{}, grad_weights{}, grad_bias{};
  bool rows16 = false, weights16 = false, grads16 = false;  // every rank's buffer starts on 16 bytes
  char* scratch = nullptr;     // the plan's parts of the workspace
  bool log_plan = false;       // each product's form to stderr
  hipStream_t stream = nullptr;
  int num_cus = 0;
};

// What the products keep in the workspace, by the shape alone.
struct ProductPlan {
  // Rows are copied with a stride of whole 16-byte vectors (ldh, ldf; else
  // the plain width) where their width is no multiple of that and the
  // product is large enough to pay for it.
  bool pack_hidden = false, pack_features = false;
  uint32_t ldh = 0, ldf = 0;
  uint32_t splits = 1;  // of the rows of an expert, for the weights' gradient
  uint32_t chunk = 0;   // rows of a partial sum of the bias's gradient
  uint32_t slots = 0;   // partial sums of a rank: every expert's rows start one of their own
  // Offsets in the scratch, and its size for the forward product and for the gradients.
  size_t rows = 0, weights = 0, forward = 0;
  size_t dz = 0, sums = 0, parts = 0, grad_rows = 0, grad_weights = 0, grads = 0;
};
ProductPlan product_plan(int dtype, uint32_t nranks, uint32_t per_rank, uint32_t capacity, uint32_t hidden,
                         uint32_t features);

hipError_t run_expert_matmul(const ProductCall& c);
hipError_t run_expert_matmul_grad(const ProductCall& c);

}  // namespace ccl
