// Verification of greedy drafts by sampling at a temperature ("Attention
// Drift", section 2: rejection sampling against the target's own distribution,
// the longest valid prefix accepted).
//
// The drafts are greedy, so their distribution is a point mass: draft x after
// row j is accepted with probability p_j(x), and a rejected one leaves the
// residual max(p_j - q, 0) = p_j without x.  A token from p_a (or from p_a without
// x) is argmax_v(l_v / T + g_v) for standard Gumbel noise g (over v != x): the
// normaliser of p does not enter, so only the acceptance tests need the row sums.
//
//   row kernel      one CTA per row: the largest logit m and the sum s of
//                   exp((l - m) / T); for a greedy request (T = 0) the argmax key.
//   request kernel  one CTA per request: the accepted prefix, then the race over
//                   the one row the next token comes from.
#include <cmath>

#include "pe_common.cuh"
#include "pe_paged.h"

namespace pe {
namespace {

constexpr int kThreads = 256;
constexpr int kWsHeader = 256;  // status word, then per row: (m, s) or the key

struct VerifyArgs {
  int B, T, V;
  const int32_t* qsl;
  const int32_t* tok;
  const void* logits;
  const float* temperature;
  const float* u;
  const float* gumbel;
  int32_t* accepted;
  int32_t* bonus;
  float* p_draft;
  uint32_t* status;
  uint64_t* rows;
};

PE_DEV float temperature_of(const VerifyArgs& a, int r) {
  const float t = a.temperature ? a.temperature[r] : 1.f;
  return t > 0.f ? t : 0.f;
}

template <typename T>
PE_DEV float logit(const VerifyArgs& a, int64_t row, int v) {
  return Elem<T>::to_f(static_cast<const T*>(a.logits)[row * a.V + v]);
}

// 1 / T, finite for every T > 0 (so that a difference of 0 stays 0)
PE_DEV float inv_temperature(float temp) { return fminf(1.f / temp, 3.0e38f); }

// probability of token v given a row's statistics (m: largest logit, s: sum of
// exp((l - m) / T)), 0 for a row without a distribution.  64 bits: one value per
// draft, and a draft is accepted by a comparison with it.
template <typename T>
PE_DEV float prob(const VerifyArgs& a, int64_t row, int v, float temp, float m, float s) {
  if (!(fabsf(m) < INFINITY)) return 0.f;
  const double d = static_cast<double>(logit<T>(a, row, v)) - static_cast<double>(m);
  return static_cast<float>(exp(d / static_cast<double>(temp)) / static_cast<double>(s));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sampled_row_kernel(const VerifyArgs a) {
  __shared__ float sm[kThreads / 32], ss[kThreads / 32];
  __shared__ uint64_t sk[kThreads / 32];
  __shared__ int req_sh;
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (row == 0 && tid == 0) *a.status = 0u;  // only the request kernel sets bits
  if (tid == 0) req_sh = -1;
  __syncthreads();
  for (int r = tid; r < a.B; r += kThreads) {
    const RowRange x = request_rows(a.qsl, r, a.T);
    if (x.q0 <= row && row < x.q1) atomicMax(&req_sh, r);
  }
  __syncthreads();
  if (req_sh < 0) return;
  const float temp = temperature_of(a, req_sh);
  if (temp == 0.f) {
    unsigned long long k = 0ull;
    for (int v = tid; v < a.V; v += kThreads)
      k = max(k, argmax_key(logit<T>(a, row, v), static_cast<uint32_t>(v)));
    k = warp_max_u64(k);
    if (lane == 0) sk[warp] = k;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kThreads / 32; ++w) k = max(k, static_cast<unsigned long long>(sk[w]));
      a.rows[row] = k;
    }
    return;
  }
  const float it = inv_temperature(temp);
  float m = -INFINITY, s = 0.f;
  bool nan = false;
  for (int v = tid; v < a.V; v += kThreads) {
    const float x = logit<T>(a, row, v);
    nan |= x != x;
    if (x > m) {
      s = m == -INFINITY ? 0.f : s * expf((m - x) * it);
      m = x;
    }
    if (x != -INFINITY) s += expf((x - m) * it);
  }
  const float wm = __any_sync(0xffffffffu, nan) ? NAN : warp_max(m);
  s = m == -INFINITY ? 0.f : s * expf((m - wm) * it);
  s = warp_sum(s);
  if (lane == 0) {
    sm[warp] = wm;
    ss[warp] = s;
  }
  __syncthreads();
  if (tid == 0) {
    float M = sm[0];
    for (int w = 1; w < kThreads / 32; ++w) M = (sm[w] != sm[w] || M != M) ? NAN : fmaxf(M, sm[w]);
    float S = 0.f;
    for (int w = 0; w < kThreads / 32; ++w)
      if (sm[w] != -INFINITY) S += ss[w] * expf((sm[w] - M) * it);
    a.rows[row] = (static_cast<uint64_t>(__float_as_uint(M)) << 32) | __float_as_uint(S);
  }
}

// order of a score, larger first; -inf and NaN never win (key 0)
PE_DEV unsigned long long score_order(double x) {
  if (!(x > -INFINITY)) return 0ull;
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x + 0.0));
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sampled_request_kernel(const VerifyArgs a) {
  __shared__ int bad_sh;
  __shared__ unsigned long long key_sh[kThreads / 32];
  __shared__ int idx_sh[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const RowRange x = request_rows(a.qsl, r, a.T);
  const int n = x.q1 - x.q0;
  uint32_t st = x.bad ? PE_ST_ROWS_RANGE : 0u;
  const float t0 = a.temperature ? a.temperature[r] : 1.f;
  if (!(t0 >= 0.f)) st |= PE_ST_SAMPLING;
  const float temp = temperature_of(a, r);
  if (tid == 0) bad_sh = n;
  __syncthreads();
  // draft j follows row j - 1
  for (int j = 1 + tid; j < n; j += kThreads) {
    const int64_t row = x.q0 + j - 1;
    const int v = a.tok[row + 1];
    const uint64_t w = a.rows[row];
    float p = 0.f;
    if (v < 0 || v >= a.V) {
      st |= PE_ST_TOKEN_RANGE;
    } else if (temp == 0.f) {
      p = static_cast<uint32_t>(v) == ~static_cast<uint32_t>(w) ? 1.f : 0.f;
    } else {
      p = prob<T>(a, row, v, temp, __uint_as_float(static_cast<uint32_t>(w >> 32)),
                  __uint_as_float(static_cast<uint32_t>(w)));
    }
    if (a.p_draft) a.p_draft[row + 1] = p;
    if (temp == 0.f ? p == 0.f : !(a.u[row + 1] < p)) atomicMin(&bad_sh, j - 1);
  }
  if (tid == 0 && n > 0 && a.p_draft) a.p_draft[x.q0] = 1.f;
  __syncthreads();
  const int acc = n > 0 ? min(bad_sh, n - 1) : 0;
  int bonus = -1;
  if (n > 0) {
    const int64_t row = x.q0 + acc;
    const uint64_t w = a.rows[row];
    if (temp == 0.f) {
      bonus = static_cast<int>(~static_cast<uint32_t>(w));
    } else {
      const float m = __uint_as_float(static_cast<uint32_t>(w >> 32));
      if (fabsf(m) < INFINITY) {
        const int skip = acc + 1 < n ? a.tok[row + 1] : -1;
        unsigned long long best = 0ull;
        int bi = 0x7fffffff;
        for (int v = tid; v < a.V; v += kThreads) {
          const float l = logit<T>(a, row, v);
          if (v == skip || l == -INFINITY) continue;
          const double s = static_cast<double>(l) / temp + a.gumbel[static_cast<int64_t>(r) * a.V + v];
          const unsigned long long k = score_order(s);
          if (k > best) {
            best = k;
            bi = v;
          }
        }
        for (int o = 16; o; o >>= 1) {
          const unsigned long long k2 = __shfl_xor_sync(0xffffffffu, best, o);
          const int b2 = __shfl_xor_sync(0xffffffffu, bi, o);
          if (k2 > best || (k2 == best && b2 < bi)) {
            best = k2;
            bi = b2;
          }
        }
        if (lane == 0) {
          key_sh[warp] = best;
          idx_sh[warp] = bi;
        }
        __syncthreads();
        if (tid == 0)
          for (int i = 1; i < kThreads / 32; ++i)
            if (key_sh[i] > best || (key_sh[i] == best && idx_sh[i] < bi)) {
              best = key_sh[i];
              bi = idx_sh[i];
            }
        bonus = best ? bi : -1;
      } else {
        st |= PE_ST_SAMPLING;
      }
    }
  }
  if (tid == 0) {
    a.accepted[r] = acc;
    a.bonus[r] = bonus;
  }
  if (st) set_status(a.status, st);
}

}  // namespace
}  // namespace pe

using namespace pe;

extern "C" size_t pe_verify_sampled_workspace_bytes(int max_batch, int max_rows_in, int vocab) {
  if (max_batch < 0 || max_rows_in < 0 || vocab < 1) return 0;
  return static_cast<size_t>(kWsHeader) + static_cast<size_t>(max_rows_in) * 8;
}

extern "C" int pe_verify_sampled(int B, int T_in, const int32_t* qsl, const int32_t* tok,
                                 const void* logits, int vocab, int dtype,
                                 const float* temperature, const float* u, const float* gumbel,
                                 int32_t* accepted, int32_t* bonus, float* p_draft, void* ws,
                                 size_t ws_bytes, void* stream) {
  NvtxRange nvtx("pe_verify_sampled");
  if (B < 0 || T_in < 0 || vocab < 1) return PE_ERR_ARG;
  if (dtype != PE_DTYPE_F32 && dtype != PE_DTYPE_BF16) return PE_ERR_UNSUPPORTED;
  if (B == 0) return T_in == 0 ? PE_OK : PE_ERR_ARG;
  if (B > 65535) return PE_ERR_UNSUPPORTED;
  if (!qsl || !accepted || !bonus || !ws) return PE_ERR_ARG;
  if (T_in > 0 && (!tok || !logits || !u || !gumbel)) return PE_ERR_ARG;
  const int esize = dtype == PE_DTYPE_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % esize != 0) return PE_ERR_ARG;
  for (const void* p : {static_cast<const void*>(qsl), static_cast<const void*>(tok),
                        static_cast<const void*>(temperature), static_cast<const void*>(u),
                        static_cast<const void*>(gumbel), static_cast<const void*>(accepted),
                        static_cast<const void*>(bonus), static_cast<const void*>(p_draft)})
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return PE_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(ws) % 256 != 0) return PE_ERR_ARG;
  if (ws_bytes < pe_verify_sampled_workspace_bytes(B, T_in, vocab)) return PE_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  VerifyArgs a = {B, T_in, vocab, qsl, tok, logits, temperature, u, gumbel, accepted, bonus, p_draft,
                  static_cast<uint32_t*>(ws),
                  reinterpret_cast<uint64_t*>(static_cast<char*>(ws) + kWsHeader)};
  const bool f32 = dtype == PE_DTYPE_F32;
  if (T_in > 0) {
    if (launch_pdl(f32 ? sampled_row_kernel<float> : sampled_row_kernel<bf16>, dim3(T_in),
                   dim3(kThreads), 0, st, a) != cudaSuccess)
      return PE_ERR_CUDA;
  } else if (cudaMemsetAsync(ws, 0, sizeof(uint32_t), st) != cudaSuccess) {
    return PE_ERR_CUDA;
  }
  return launch_pdl(f32 ? sampled_request_kernel<float> : sampled_request_kernel<bf16>, dim3(B),
                    dim3(kThreads), 0, st, a) == cudaSuccess
             ? PE_OK
             : PE_ERR_CUDA;
}
