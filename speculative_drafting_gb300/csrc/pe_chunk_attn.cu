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
// keys.  One CTA of four warps per (row, query head); a warp takes every fourth group of
// 32 keys.  For the scores a lane owns a key (one reduction over the warp per group, not
// per key); for P V a lane owns every 32nd dimension.  fp32 throughout.
#include "pe_common.cuh"
#include "pe_paged.h"

namespace pe {
namespace {

constexpr int kWarps = 4;

// sum over a 16-byte vector of k times q
template <typename T>
PE_DEV float dot16(const uint4& k, const float* q, float acc) {
  constexpr int kVec = 16 / sizeof(T);
  float f[kVec];
  unpack16<T>(k, f);
#pragma unroll
  for (int i = 0; i < kVec; ++i) acc = fmaf(f[i], q[i], acc);
  return acc;
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) chunk_simt_kernel(const ChunkArgs a) {
  constexpr int kVec = 16 / sizeof(T);
  __shared__ __align__(16) float q_sh[128];
  __shared__ float wm[kWarps], wl[kWarps], wacc[kWarps][128];
  __shared__ int req_sh;
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const T* q = static_cast<const T*>(a.q) + row * a.ld_q + static_cast<int64_t>(h) * a.hd;
  // the request of this row: the last one that starts at or before it
  if (tid == 0) req_sh = -1;
  if (tid < a.hd) q_sh[tid] = Elem<T>::to_f(q[tid]) / sqrtf(static_cast<float>(a.hd));
  __syncthreads();
  for (int r = tid; r < a.B; r += 32 * kWarps) {
    const RowRange x = request_rows(a.qsl, r, a.T);
    if (x.bad) set_status(a.status, PE_ST_ROWS_RANGE);
    if (x.q0 <= row && row < x.q1) atomicMax(&req_sh, r);
  }
  __syncthreads();
  const int r = req_sh;
  if (r < 0) return;  // behind the last request
  const RowRange rr = request_rows(a.qsl, r, a.T);
  const int n = rr.q1 - rr.q0, j = row - rr.q0;
  const int64_t Lmax = static_cast<int64_t>(a.max_blocks) * a.bs;
  int L = a.seq_len[r];
  if (L < 0 || L > Lmax) {
    if (tid == 0) set_status(a.status, PE_ST_BLOCK_RANGE);
    L = static_cast<int>(min(max(static_cast<int64_t>(L), int64_t{0}), Lmax));
  }
  const int lim = L - n + j;  // the row's own position
  const int g = h / (a.H / a.G);
  const T* kc = static_cast<const T*>(a.k_cache);
  const T* vc = static_cast<const T*>(a.v_cache);
  float m = -INFINITY, l = 0.f;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t t0 = 32 * warp; t0 <= lim; t0 += 32 * kWarps) {
    // scores: this lane's key
    const int t = static_cast<int>(t0) + lane;
    int64_t base = -1;
    float s = -INFINITY;
    if (t0 + lane <= lim) {
      const int blk = a.block_table[static_cast<int64_t>(r) * a.max_blocks + t / a.bs];
      if (blk < 0 || blk >= a.num_blocks) {
        set_status(a.status, PE_ST_BLOCK_RANGE);
      } else {
        base = ((static_cast<int64_t>(blk) * a.G + g) * a.bs + t % a.bs) * a.hd;
        const uint4* k = reinterpret_cast<const uint4*>(kc + base);
        s = 0.f;
#pragma unroll 4
        for (int i = 0; i < a.hd / kVec; ++i) s = dot16<T>(k[i], q_sh + i * kVec, s);
      }
    }
    const float mn = fmaxf(m, warp_max(s));
    const float al = m == -INFINITY ? 1.f : expf(m - mn);
    // (a NaN score stays NaN; a key that is not there has weight 0)
    const float p = base < 0 ? 0.f : expf(s - (mn == -INFINITY ? 0.f : mn));
    l = l * al + warp_sum(p);
    m = mn;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] *= al;
    // P V: the keys that are there, four at a time
    unsigned todo = __ballot_sync(0xffffffffu, base >= 0);
    while (todo) {
      float v[4][4], pj[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int src = todo ? __ffs(todo) - 1 : 0;
        const bool ok = todo != 0;
        todo &= todo - 1;
        pj[x] = __shfl_sync(0xffffffffu, p, src);
        const int64_t b = __shfl_sync(0xffffffffu, base, src);
        if (!ok) pj[x] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[x][i] = ok && lane + 32 * i < a.hd ? Elem<T>::to_f(vc[b + lane + 32 * i]) : 0.f;
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(pj[x], v[x][i], acc[i]);
    }
  }
  if (lane == 0) {
    wm[warp] = m;
    wl[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < a.hd) wacc[warp][lane + 32 * i] = acc[i];
  __syncthreads();
  // a sink logit joins the maximum and the denominator (its value row is zero); a warp
  // that saw no key has l = 0 (NaN: it saw one)
  const float sk = a.sink ? a.sink[h] : -INFINITY;
  float M = sk;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w]);
  auto weight = [&](int w) { return wl[w] == 0.f ? 0.f : wm[w] == -INFINITY ? wl[w] : expf(wm[w] - M); };
  float den = sk == -INFINITY ? 0.f : expf(sk - M);
  bool any = false;
  for (int w = 0; w < kWarps; ++w) {
    den += weight(w) * wl[w];
    any |= wl[w] != 0.f;
  }
  T* out = static_cast<T*>(a.out) + row * a.ld_out + static_cast<int64_t>(h) * a.hd;
  for (int d = tid; d < a.hd; d += 32 * kWarps) {
    float num = 0.f;
    for (int w = 0; w < kWarps; ++w) num += weight(w) * wacc[w][d];
    out[d] = Elem<T>::from_f(any ? num / den : 0.f);
  }
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

extern "C" int pe_chunk_attention(const pe_attn_plan* plan, int B, int T, const int32_t* qsl,
                                  const int32_t* seq_len, const void* q, int64_t ld_q,
                                  const void* k_cache, const void* v_cache,
                                  const int32_t* block_table, int max_blocks, int num_blocks,
                                  const float* sink, void* out, int64_t ld_out, void* ws,
                                  size_t ws_bytes, void* stream) {
  NvtxRange nvtx("pe_chunk_attention");
  if (!plan_ok(plan) || B < 0 || T < 0 || max_blocks < 1 || num_blocks < 0) return PE_ERR_ARG;
  const int64_t width = static_cast<int64_t>(plan->n_heads) * plan->head_dim;
  if (ld_q < width || ld_out < width || ld_q % 8 || ld_out % 8) return PE_ERR_ARG;
  if (B > 65535 || static_cast<int64_t>(T) * plan->n_heads > 0x7fffffff ||
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
  if (chunk_tc_takes(plan) && num_blocks > 0) return launch_chunk_tc(a, static_cast<char*>(ws), st);
  const dim3 grid(static_cast<unsigned>(T), static_cast<unsigned>(plan->n_heads));
  const cudaError_t e = plan->dtype == PE_DTYPE_BF16
                            ? launch_chained(chunk_simt_kernel<bf16>, grid, dim3(32 * kWarps), 0, st, a)
                            : launch_chained(chunk_simt_kernel<float>, grid, dim3(32 * kWarps), 0, st, a);
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}
