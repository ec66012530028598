// Attention of each request's new rows over its pages (pe_chunk_attention).
//
// Row j of request r stands at position L_r - n_r + j and sees every cache
// position up to its own:
//   o = sum_t p_t v_t,  p_t = exp(s_t - m) / (sum_t exp(s_t - m) + exp(sink - m)),
//   s_t = q . k_t / sqrt(hd),
// computed in one pass over the keys with a running maximum and sum.
//
// This file: the entry point, and the kernel of the shapes that the tensor-core kernels
// (pe_chunk_attn_tc.cu) do not take: fp32 plans, and blocks that are no multiple of 8
// keys.  One CTA per (row, query head).
#include "pe_attn_row.cuh"
#include "pe_testing.h"

namespace pe {
namespace {

// (48 registers: with 56 a small fp32 call takes 17 us, with 48 13 us, with 40 16 us)
template <typename T>
__global__ void __launch_bounds__(32 * kRowWarps, 10) chunk_simt_kernel(const ChunkArgs a) {
  __shared__ RowScratch sh;
  __shared__ int req_sh;
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  // the request of this row: the last one that starts at or before it
  if (tid == 0) req_sh = -1;
  // (rows behind the last request are not read: they may not be written yet)
  if (row < a.qsl[a.B]) row_query<T>(a, row, h, sh);
  __syncthreads();
  const int64_t Lmax = static_cast<int64_t>(a.max_blocks) * a.bs;
  for (int r = tid; r < a.B; r += 32 * kRowWarps) {
    const RowRange x = request_rows(a.qsl, r, a.T);
    if (x.bad) set_status(a.status, PE_ST_ROWS_RANGE);
    // (of every request, those without rows too)
    if (row == 0 && h == 0 && (a.seq_len[r] < 0 || a.seq_len[r] > Lmax)) set_status(a.status, PE_ST_BLOCK_RANGE);
    if (x.q0 <= row && row < x.q1) atomicMax(&req_sh, r);
  }
  __syncthreads();
  const int r = req_sh;
  if (r < 0) return;  // behind the last request
  const RowRange rr = request_rows(a.qsl, r, a.T);
  const int n = rr.q1 - rr.q0, j = row - rr.q0;
  const int L = static_cast<int>(min(max(static_cast<int64_t>(a.seq_len[r]), int64_t{0}), Lmax));
  const int lim = L - n + j;  // the row's own position
  attend_row<T>(a, r, row, h, lim, sh);
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace
}  // namespace pe

using namespace pe;

extern "C" size_t pe_chunk_attention_workspace_bytes(const pe_attn_plan* plan, int max_batch,
                                                     int max_rows) {
  if (!plan_ok(plan) || max_batch < 0 || max_rows < 0) return 0;
  return chunk_tc_takes(plan) ? chunk_tc_workspace(plan, max_rows) : 256;
}

namespace {

int chunk_attention(const pe_attn_plan* plan, int B, int T, const int32_t* qsl, const int32_t* seq_len,
                    const void* q, int64_t ld_q, const void* k_cache, const void* v_cache,
                    const int32_t* block_table, int max_blocks, int num_blocks, const float* sink, void* out,
                    int64_t ld_out, void* ws, size_t ws_bytes, void* stream, int stall) {
  if (!plan_ok(plan) || B < 0 || T < 0 || max_blocks < 1 || num_blocks < 0) return PE_ERR_ARG;
  const int64_t width = static_cast<int64_t>(plan->n_heads) * plan->head_dim;
  if (ld_q < width || ld_out < width || ld_q % 8 || ld_out % 8) return PE_ERR_ARG;
  if (B > 65535 || static_cast<int64_t>(T) * plan->n_heads > 0x7fffff00 ||
      static_cast<int64_t>(max_blocks) * plan->block_size > 0x7fffff00)
    return PE_ERR_UNSUPPORTED;
  if (static_cast<double>(num_blocks) * plan->n_kv_heads * plan->block_size >= 2147483648.0)
    return PE_ERR_UNSUPPORTED;
  if (!ws || !aligned(ws, 256) || ws_bytes < pe_chunk_attention_workspace_bytes(plan, B, T))
    return PE_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (B > 0 && T > 0) {
    if (!qsl || !seq_len || !q || !k_cache || !v_cache || !block_table || !out) return PE_ERR_ARG;
    for (const void* p : {q, k_cache, v_cache, static_cast<const void*>(out)})
      if (!aligned(p, 16)) return PE_ERR_ARG;
    if (!aligned(qsl, 4) || !aligned(seq_len, 4) || !aligned(block_table, 4) || !aligned(sink, 4))
      return PE_ERR_ARG;
  }
  if (B == 0 || T == 0) return PE_OK;
  ChunkArgs a = {};
  a.B = B;
  a.T = T;
  a.H = plan->n_heads;
  a.G = plan->n_kv_heads;
  a.hd = plan->head_dim;
  a.bs = plan->block_size;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.qsl = qsl;
  a.seq_len = seq_len;
  a.q = q;
  a.ld_q = ld_q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table;
  a.sink = sink;
  a.out = out;
  a.ld_out = ld_out;
  a.status = static_cast<uint32_t*>(ws);
  a.stall = stall;
  if (chunk_tc_takes(plan) && num_blocks > 0) return launch_chunk_tc(a, static_cast<char*>(ws), st);
  const dim3 grid(static_cast<unsigned>(T), static_cast<unsigned>(plan->n_heads));
  const cudaError_t e = plan->dtype == PE_DTYPE_BF16
                            ? launch_chained(chunk_simt_kernel<bf16>, grid, dim3(32 * kRowWarps), 0, st, a)
                            : launch_chained(chunk_simt_kernel<float>, grid, dim3(32 * kRowWarps), 0, st, a);
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}

}  // namespace

extern "C" int pe_chunk_attention(const pe_attn_plan* plan, int B, int T, const int32_t* qsl,
                                  const int32_t* seq_len, const void* q, int64_t ld_q,
                                  const void* k_cache, const void* v_cache,
                                  const int32_t* block_table, int max_blocks, int num_blocks,
                                  const float* sink, void* out, int64_t ld_out, void* ws,
                                  size_t ws_bytes, void* stream) {
  NvtxRange nvtx("pe_chunk_attention");
  return chunk_attention(plan, B, T, qsl, seq_len, q, ld_q, k_cache, v_cache, block_table, max_blocks,
                         num_blocks, sink, out, ld_out, ws, ws_bytes, stream, 0);
}

extern "C" int pe_test_chunk_attention_stall(const pe_attn_plan* plan, int slot, int B, int T, const int32_t* qsl,
                                             const int32_t* seq_len, const void* q, int64_t ld_q,
                                             const void* k_cache, const void* v_cache,
                                             const int32_t* block_table, int max_blocks, int num_blocks,
                                             const float* sink, void* out, int64_t ld_out, void* ws,
                                             size_t ws_bytes, void* stream) {
  if (slot < 0 || slot > 7) return PE_ERR_ARG;
  return chunk_attention(plan, B, T, qsl, seq_len, q, ld_q, k_cache, v_cache, block_table, max_blocks,
                         num_blocks, sink, out, ld_out, ws, ws_bytes, stream, 1 + slot);
}
