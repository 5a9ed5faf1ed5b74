// The optimizer's table of tensors, as spec_adamw_table lays it out.
#pragma once

#include "draft.cuh"

namespace sv {

constexpr int AD_ITEM = 4096;        // elements of a work item
constexpr uint32_t AD_MAGIC = 0x41644d57u;

struct AdTensor {
  void *param;
  const void *grad;
  void *m, *v;
  float *ms, *vs;
  float *master;
  long long n;
  int bf16;      // weight and gradient type
  int vec;       // every pointer suits 16-byte vectors
};
static_assert(sizeof(AdTensor) == 72, "table layout");

struct AdHeader {      // first 64 bytes of a table
  uint32_t magic;
  int n_tensors;
  long long n_items;
  int state_bits;
  int pad[11];
};
static_assert(sizeof(AdHeader) == 64, "table layout");

struct AdItem {
  int tensor;
  int chunk;   // element offset / AD_ITEM
};

}  // namespace sv
