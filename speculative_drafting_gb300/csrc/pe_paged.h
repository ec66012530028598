// Host-side checks and launch interfaces of the paged attention calls.
#pragma once

#include "pe_internal.h"

namespace pe {

// launch_pdl with the carveout as a launch attribute: no function attribute call per
// launch (a microsecond of host time in a small call).
template <typename... Exp, typename... Act>
inline cudaError_t launch_chained(void (*kernel)(Exp...), dim3 grid, dim3 block, size_t smem,
                                  cudaStream_t st, Act&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
  attr[1].val.sharedMemCarveout = cudaSharedmemCarveoutMaxShared;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Act&&>(args)...);
}

// Whether pe_attn_plan_init filled this plan (its shape fields are in range).
bool plan_ok(const pe_attn_plan* p);

// One call of pe_chunk_attention or pe_tree_attention, as their kernels take it.
struct ChunkArgs {
  int B, T, H, G, hd, bs, max_blocks, num_blocks;
  const int32_t* qsl;
  const int32_t* seq_len;
  const void* q;
  int64_t ld_q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_table;
  const float* sink;
  void* out;
  int64_t ld_out;
  uint32_t* status;
  int stall;  // pe_test_chunk_attention_stall's, else 0
};
// The masks of pe_tree_attention beside it (an argument of their own: in ChunkArgs they cost the
// kernels without a tree half a microsecond of a small call, in registers).
struct TreeMask {
  const uint32_t* bits;  // [T][words], null: no tree
  int words;
};

// The tensor-core kernels of the two (bf16, blocks of a multiple of 8 keys).
bool chunk_tc_takes(const pe_attn_plan* plan);
size_t chunk_tc_workspace(const pe_attn_plan* plan, int max_rows);
int launch_chunk_tc(const ChunkArgs& a, const TreeMask& mask, char* ws, cudaStream_t st);

// Rows [q0, q1) of request r, clamped to [0, T]; bad: qsl is not a
// non-decreasing run from 0 to at most T.
struct RowRange {
  int q0, q1;
  bool bad;
};
__device__ __forceinline__ RowRange row_range(int a, int b, int r, int T) {  // a, b: qsl[r], qsl[r + 1]
  RowRange x;
  x.bad = a < 0 || b > T || b < a || (r == 0 && a != 0);
  x.q0 = min(max(a, 0), T);
  x.q1 = min(max(b, x.q0), T);
  return x;
}
__device__ __forceinline__ RowRange request_rows(const int32_t* qsl, int r, int T) {
  return row_range(qsl[r], qsl[r + 1], r, T);
}

}  // namespace pe
