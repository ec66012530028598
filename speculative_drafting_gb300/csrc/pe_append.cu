// Norm of the query and key heads, position rotation and paged cache write of
// the rows of one QKV projection ("P-EAGLE: parallel speculative decoding in
// vLLM", KV cache and CUDA graphs: slots address the paged cache, and rows with
// PADDING_SLOT_ID = -1 are not written).
//
//   y = x * gamma / sqrt(mean(x^2) + eps)                (q and k heads, optional)
//   (y_i, y_{i+hd/2}) -> (y_i c - y_{i+hd/2} s, y_{i+hd/2} c + y_i s),
//   c, s = cos, sin of pos * theta^(-2i/hd)              (q and k heads)
//
// Everything is fp32 until the one rounding of the result.
//
//   append_kernel       bf16 with head size 64 or 128 (and fp32 with the same): 16-byte
//                       vectors.  A CTA walks rows and forms a row's cos and sin once,
//                       in shared memory.
//   append_any_kernel   every other head size: one warp per (row, head).
#include <algorithm>
#include <cmath>

#include "pe_common.cuh"
#include "pe_paged.h"

namespace pe {
namespace {

constexpr int kWarps = 4;    // per CTA
constexpr int kRowCtas = 7;  // append_kernel's CTAs per SM

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
  int head0, heads_per_cta;  // append_kernel: the first head, heads of a CTA's row
  uint64_t turn[64];
};

// Where head h of a row goes, or NULL: q rows without a q_out, rows without a slot.
template <typename T>
PE_DEV T* head_dst(const AppendArgs& a, int64_t t, int64_t slot, int h) {
  if (h < a.H) return a.q_out ? static_cast<T*>(a.q_out) + (t * a.H + h) * a.hd : nullptr;
  if (slot < 0) return nullptr;
  const int g = h < a.H + a.G ? h - a.H : h - a.H - a.G;
  T* cache = static_cast<T*>(h < a.H + a.G ? a.k_cache : a.v_cache);
  // 32-bit division where it is enough: a 64-bit one costs as much as the rotation
  const bool small = slot <= 0xffffffffll;
  const int64_t blk = small ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(a.bs) : slot / a.bs;
  return cache + ((blk * a.G + g) * a.bs + (slot - blk * a.bs)) * a.hd;
}

// Threads of a head: hd / 2 / kVec, each with the kVec pairs (i, i + hd/2) of one
// 16-byte vector from either half.  Every thread keeps its pairs for all the heads it
// visits.  A CTA walks rows (or slices of rows); the next vectors, and the next row's
// position, slot and table of cos and sin, are under way while the current ones are
// worked on.  Small CTAs, so that a barrier per row holds up few warps: the kernel takes
// 39.5 us for 8192 rows of 48 heads of 128 with 128 threads (5.1 TB/s), 49 us with 256, and
// 42 us with a row per warp and no barrier (fewer bytes of a row in flight).  The whole
// call takes 41 to 42 us, 37.5 without norms; a plain copy of the same bytes 33.  Slots in
// whole blocks or in order instead of at random change it by 1 us.
template <typename T, int HD>
__global__ void __launch_bounds__(32 * kWarps, kRowCtas)
    append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kVec = 16 / sizeof(T);
  constexpr int kHalf = HD / 2;
  constexpr int kLanes = kHalf / kVec;   // threads per head
  constexpr int kHeads = 32 * kWarps / kLanes;  // heads per round
  __shared__ __align__(16) float cs[2][kHalf], sn[2][kHalf];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, sub = tid % kLanes;
  const int h_lo = a.head0 + blockIdx.y * a.heads_per_cta;
  const int h0 = h_lo + tid / kLanes, h_end = min(h_lo + a.heads_per_cta, a.H + 2 * a.G);
  const int64_t slots = static_cast<int64_t>(a.num_blocks) * a.bs;
  auto vec = [&](int64_t t, int h, int half) {
    const T* x = static_cast<const T*>(a.qkv) + t * a.ld_qkv + static_cast<int64_t>(h) * HD;
    return *reinterpret_cast<const uint4*>(x + half * kHalf + sub * kVec);
  };
  auto table = [&](int64_t pos, int buf) {
    if (tid < kHalf) rope_cos_sin(pos, a.turn[tid], cs[buf][tid], sn[buf][tid]);
  };
  int64_t t = blockIdx.x;
  int64_t slot = a.slot[t];
  uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
  if (h0 < h_end) {
    lo = vec(t, h0, 0);
    hi = vec(t, h0, 1);
  }
  table(a.pos[t], 0);
  for (int buf = 0; t < a.T; buf ^= 1) {
    const int64_t tn = t + gridDim.x;
    int64_t pos_n = 0, slot_n = -1;
    if (tn < a.T) {
      pos_n = a.pos[tn];
      slot_n = a.slot[tn];
    }
    if (slot >= slots) {
      if (tid == 0) set_status(a.status, PE_ST_BLOCK_RANGE);
      slot = -1;
    }
    __syncthreads();  // this row's table; the table before is no longer read
    float c[kVec], s[kVec];
#pragma unroll
    for (int i = 0; i < kVec; i += 4) {
      *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(&cs[buf][sub * kVec + i]);
      *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(&sn[buf][sub * kVec + i]);
    }
    for (int hb = h_lo; hb < h_end; hb += kHeads) {
      const int h = hb + tid / kLanes;  // the last round may be short: h >= h_end has no work
      const uint4 l4 = lo, h4 = hi;
      const bool same = hb + kHeads < h_end;
      const int hn = same ? h + kHeads : h0;
      if ((same || tn < a.T) && hn < h_end) {
        lo = vec(same ? t : tn, hn, 0);
        hi = vec(same ? t : tn, hn, 1);
      }
      float p[kVec], q[kVec];
      unpack16<T>(l4, p);
      unpack16<T>(h4, q);
      const T* gain = static_cast<const T*>(h < a.H ? a.gamma_q : a.gamma_k);
      const bool turns = h < a.H + a.G;
      // (the same for every thread, for the shuffles)
      if (a.gamma_q || a.gamma_k) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          ss = fmaf(p[i], p[i], ss);
          ss = fmaf(q[i], q[i], ss);
        }
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (gain && turns) {
          const float inv = 1.0f / sqrtf(ss / static_cast<float>(HD) + a.eps);
          float g0[kVec], g1[kVec];
          unpack16<T>(*reinterpret_cast<const uint4*>(gain + sub * kVec), g0);
          unpack16<T>(*reinterpret_cast<const uint4*>(gain + kHalf + sub * kVec), g1);
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            p[i] *= inv * g0[i];
            q[i] *= inv * g1[i];
          }
        }
      }
      uint4 o0 = l4, o1 = h4;
      if (turns) {
        float y[kVec], z[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          y[i] = p[i] * c[i] - q[i] * s[i];
          z[i] = q[i] * c[i] + p[i] * s[i];
        }
        o0 = pack16<T>(y);
        o1 = pack16<T>(z);
      }
      T* dst = h < h_end ? head_dst<T>(a, t, slot, h) : nullptr;
      if (dst) {
        *reinterpret_cast<uint4*>(dst + sub * kVec) = o0;
        *reinterpret_cast<uint4*>(dst + kHalf + sub * kVec) = o1;
      }
    }
    if (tn < a.T) table(pos_n, buf ^ 1);
    t = tn;
    slot = slot_n;
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) append_any_kernel(const __grid_constant__ AppendArgs a) {
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = a.H + 2 * a.G, half = a.hd / 2;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t t = item / heads;
  if (t >= a.T) return;
  const int h = static_cast<int>(item - t * heads);
  const T* x = static_cast<const T*>(a.qkv) + t * a.ld_qkv + static_cast<int64_t>(h) * a.hd;
  int64_t slot = a.slot[t];
  if (slot >= static_cast<int64_t>(a.num_blocks) * a.bs) {
    if (lane == 0) set_status(a.status, PE_ST_BLOCK_RANGE);
    slot = -1;
  }
  T* dst = head_dst<T>(a, t, slot, h);
  if (!dst) return;
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
  if (!p || p->n_heads < 1 || p->n_heads > 65535 || p->n_kv_heads < 1 || p->n_heads % p->n_kv_heads ||
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = plan->dtype == PE_DTYPE_BF16;
  if (a.hd == 64 || a.hd == 128) {
    // Without q_out only the k and v heads are read.  A row is one CTA's, or, while the
    // rows leave SMs idle, up to four CTAs'.
    a.head0 = q_out ? 0 : a.H;
    const int n = heads - a.head0;
    const int cut = T >= 256 ? 1 : T >= 128 ? 2 : 4;
    a.heads_per_cta = (n + cut - 1) / cut;
    const int sms = num_sms_of_current_device();
    if (sms <= 0) return PE_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>(std::min(T, kRowCtas * sms)),
                    static_cast<unsigned>((n + a.heads_per_cta - 1) / a.heads_per_cta));
    auto* kernel = bf ? (a.hd == 64 ? append_kernel<bf16, 64> : append_kernel<bf16, 128>)
                      : (a.hd == 64 ? append_kernel<float, 64> : append_kernel<float, 128>);
    return launch_chained(kernel, grid, dim3(32 * kWarps), 0, st, a) == cudaSuccess ? PE_OK : PE_ERR_CUDA;
  }
  const int64_t grid = (static_cast<int64_t>(T) * heads + kWarps - 1) / kWarps;
  if (grid > 0x7fffffff) return PE_ERR_UNSUPPORTED;
  // bf16 plans have head size 64 or 128
  return launch_chained(append_any_kernel<float>, dim3(static_cast<unsigned>(grid)), dim3(32 * kWarps), 0,
                    st, a) == cudaSuccess
             ? PE_OK
             : PE_ERR_CUDA;
}
