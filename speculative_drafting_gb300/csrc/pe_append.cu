// Norm of the query and key heads, position rotation and paged cache write of
// the rows of one QKV projection ("P-EAGLE: parallel speculative decoding in
// vLLM", KV cache and CUDA graphs: slots address the paged cache, and rows with
// PADDING_SLOT_ID = -1 are not written).
//
//   y = x * gamma / sqrt(mean(x^2) + eps)                (q and k heads, optional)
//   (y_i, y_{i+hd/2}) -> (y_i c - y_{i+hd/2} s, y_{i+hd/2} c + y_i s),
//   c, s = cos, sin of pos * theta^(-2i/hd)              (q and k heads)
//
// One warp per (row, head).  Everything is fp32 until the one rounding of the
// result.
#include <cmath>

#include "pe_common.cuh"
#include "pe_paged.h"

namespace pe {
namespace {

constexpr int kWarps = 4;

struct AppendArgs {
  int T, H, G, hd, bs, num_blocks;
  float eps;
  const void* qkv;
  int64_t ld_qkv;
  const void* gamma_q;
  const void* gamma_k;
  const int64_t* pos;
  const int64_t* slot;
  void* q_out;
  void* k_cache;
  void* v_cache;
  uint32_t* status;
  uint64_t turn[64];
};

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const __grid_constant__ AppendArgs a) {
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = a.H + 2 * a.G, half = a.hd / 2;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t t = item / heads;
  if (t >= a.T) return;
  const int h = static_cast<int>(item - t * heads);
  const T* x = static_cast<const T*>(a.qkv) + t * a.ld_qkv + static_cast<int64_t>(h) * a.hd;
  T* dst;
  if (h < a.H) {
    if (!a.q_out) return;
    dst = static_cast<T*>(a.q_out) + (t * a.H + h) * a.hd;
  } else {
    const int64_t slot = a.slot[t];
    if (slot >= static_cast<int64_t>(a.num_blocks) * a.bs) {
      if (lane == 0) set_status(a.status, PE_ST_BLOCK_RANGE);
      return;
    }
    if (slot < 0) return;
    const int g = (h - a.H) % a.G;
    T* cache = static_cast<T*>(h < a.H + a.G ? a.k_cache : a.v_cache);
    dst = cache + (((slot / a.bs) * a.G + g) * a.bs + slot % a.bs) * a.hd;
  }
  if (h >= a.H + a.G) {  // a value head: copied
    for (int i = lane; i < a.hd; i += 32) dst[i] = x[i];
    return;
  }
  float lo[2], hi[2], ss = 0.f;  // half <= 64: at most two pairs a lane
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    lo[k] = i < half ? Elem<T>::to_f(x[i]) : 0.f;
    hi[k] = i < half ? Elem<T>::to_f(x[i + half]) : 0.f;
    ss = fmaf(lo[k], lo[k], ss);
    ss = fmaf(hi[k], hi[k], ss);
  }
  const T* gain = static_cast<const T*>(h < a.H ? a.gamma_q : a.gamma_k);
  float inv = 1.f;
  if (gain) inv = 1.0f / sqrtf(warp_sum(ss) / static_cast<float>(a.hd) + a.eps);
  const int64_t pos = a.pos[t];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    if (i >= half) break;
    if (gain) {
      lo[k] *= inv * Elem<T>::to_f(gain[i]);
      hi[k] *= inv * Elem<T>::to_f(gain[i + half]);
    }
    float c, s;
    rope_cos_sin(pos, a.turn[i], c, s);
    dst[i] = Elem<T>::from_f(lo[k] * c - hi[k] * s);
    dst[i + half] = Elem<T>::from_f(hi[k] * c + lo[k] * s);
  }
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

bool plan_ok(const pe_attn_plan* p) {
  if (!p || p->n_heads < 1 || p->n_kv_heads < 1 || p->n_heads % p->n_kv_heads ||
      p->n_heads / p->n_kv_heads > 128 || p->head_dim < 8 || p->head_dim % 8 ||
      p->head_dim > 128 || p->block_size < 1 || !(p->eps >= 0.f))
    return false;
  if (p->dtype == PE_DTYPE_F32) return true;
  return p->dtype == PE_DTYPE_BF16 && (p->head_dim == 64 || p->head_dim == 128);
}

}  // namespace pe

using namespace pe;

extern "C" int pe_attn_plan_init(pe_attn_plan* plan, int n_heads, int n_kv_heads, int head_dim,
                                 int block_size, int dtype, float eps, float rope_theta) {
  if (!plan) return PE_ERR_ARG;
  pe_attn_plan p = {};
  p.n_heads = n_heads;
  p.n_kv_heads = n_kv_heads;
  p.head_dim = head_dim;
  p.block_size = block_size;
  p.dtype = dtype;
  p.eps = eps;
  *plan = pe_attn_plan{};
  if (!plan_ok(&p) || !(rope_theta > 0.f) || !std::isfinite(rope_theta) || !std::isfinite(eps))
    return PE_ERR_UNSUPPORTED;
  // frequency i, theta^(-2i/hd) radians per position, as the fraction of a turn
  // per position in 64-bit fixed point (whole turns drop out).  long double holds
  // 64 bits or more, so the angle of a position up to 2^40 is right to 4e-7 rad
  // (with the 53 bits of a double it was off by 1e-4 there).
  for (int i = 0; i < head_dim / 2; ++i) {
    const long double turn = std::pow(static_cast<long double>(rope_theta),
                                      -2.0L * static_cast<long double>(i) /
                                          static_cast<long double>(head_dim)) /
                             6.283185307179586476925286766559005768L;
    p.rope_turn[i] = static_cast<uint64_t>(std::ldexp(turn - std::floor(turn), 64));
  }
  *plan = p;
  return PE_OK;
}

extern "C" int pe_qkv_append(const pe_attn_plan* plan, int T, const void* qkv, int64_t ld_qkv,
                             const void* gamma_q, const void* gamma_k, const int64_t* pos,
                             const int64_t* slot, int num_blocks, void* q_out, void* k_cache,
                             void* v_cache, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx("pe_qkv_append");
  if (!plan_ok(plan) || T < 0 || num_blocks < 0) return PE_ERR_ARG;
  const int heads = plan->n_heads + 2 * plan->n_kv_heads;
  if (ld_qkv < static_cast<int64_t>(heads) * plan->head_dim || ld_qkv % 8) return PE_ERR_ARG;
  if (T == 0) return PE_OK;
  if (!qkv || !pos || !slot || !k_cache || !v_cache || !ws) return PE_ERR_ARG;
  for (const void* p : {qkv, gamma_q, gamma_k, static_cast<const void*>(q_out),
                        static_cast<const void*>(k_cache), static_cast<const void*>(v_cache)})
    if (!aligned(p, 16)) return PE_ERR_ARG;
  if (!aligned(pos, 8) || !aligned(slot, 8) || !aligned(ws, 256) || ws_bytes < 256)
    return PE_ERR_ARG;
  AppendArgs a = {};
  a.T = T;
  a.H = plan->n_heads;
  a.G = plan->n_kv_heads;
  a.hd = plan->head_dim;
  a.bs = plan->block_size;
  a.num_blocks = num_blocks;
  a.eps = plan->eps;
  a.qkv = qkv;
  a.ld_qkv = ld_qkv;
  a.gamma_q = gamma_q;
  a.gamma_k = gamma_k;
  a.pos = pos;
  a.slot = slot;
  a.q_out = q_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.status = static_cast<uint32_t*>(ws);
  for (int i = 0; i < 64; ++i) a.turn[i] = plan->rope_turn[i];
  const int64_t items = static_cast<int64_t>(T) * heads;
  const int64_t grid = (items + kWarps - 1) / kWarps;
  if (grid > 0x7fffffff) return PE_ERR_UNSUPPORTED;
  const cudaError_t e =
      plan->dtype == PE_DTYPE_BF16
          ? launch_pdl(append_kernel<bf16>, dim3(static_cast<unsigned>(grid)), dim3(32 * kWarps), 0,
                       static_cast<cudaStream_t>(stream), a)
          : launch_pdl(append_kernel<float>, dim3(static_cast<unsigned>(grid)), dim3(32 * kWarps), 0,
                       static_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}
