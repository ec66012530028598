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
//   row kernel      CTA (row, chunk): the chunk's largest logit m and the sum s of
//                   exp((l - m) / T); for a greedy request (T = 0) its argmax key.
//                   Streams the logits once: HBM-bound.
//   request kernel  CTA (request, chunk): joins the rows' chunks, walks the drafts
//                   to the accepted prefix, then races over its chunk of the one
//                   row that the next token comes from; the last CTA of a request
//                   to finish takes the best of the chunks.
//
// The request kernel reads one row per request a second time (1 / n of the logits)
// and its noise; racing in the row kernel instead would read the noise for every
// row.
#include <algorithm>
#include <cmath>

#include "pe_common.cuh"
#include "pe_paged.h"

namespace pe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;            // 16-byte loads in flight per thread
constexpr int kMaxChunkBytes = 65536; // of a row, per CTA of the row kernel
constexpr int kRace = 8;              // logits per thread and round of the race
constexpr int kRaceRounds = 2;        // rounds whose loads are in flight together

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
  int chunk, splits;    // row kernel
  int rchunk, rsplits;  // request kernel
  int vec;              // the race's rows are 16-byte aligned
  uint64_t* rows;       // [T][splits]: (m, s) or the argmax key
  uint32_t* done;       // [B] CTAs of the request kernel that finished
  ulonglong2* best;     // [B][rsplits]: order of the score, token
};

// as given (NULL: 1), and as used
PE_DEV float given_temperature(const VerifyArgs& a, int r) {
  return a.temperature ? __ldcg(a.temperature + r) : 1.f;
}
PE_DEV float temperature_of(float t) {
  return t > 0.f ? fminf(fmaxf(t, 1e-30f), 1e30f) : 0.f;  // 1 / T stays finite and above 0
}

PE_DEV float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
PE_DEV uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// The request of a row, by one warp: the last r with qsl[r] <= row (32 probes a
// round).  -1: the row is behind the last request.
PE_DEV int request_of(const VerifyArgs& a, int row, int lane) {
  int lo = 0, hi = a.B;  // qsl[lo] <= row < qsl[hi], were qsl[B] past every row
  if (a.qsl[a.B] <= row || a.qsl[0] > row) return -1;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < hi && a.qsl[min(at, a.B)] <= row);
    const int k = 31 - __clz(le | 1u);
    const int nlo = lo + k * step;
    hi = min(hi, nlo + step);
    lo = nlo;
  }
  return lo;
}

// Largest logit m seen and the sum s of 2^((l - m) c), c = log2(e) / T.  The difference
// is formed first: it is exact near the largest logit, whatever its size.  A NaN logit
// makes m NaN, a +inf one +inf: neither row has a distribution (nor has one of -inf
// alone).
struct Stat {
  float m, s;
};
PE_DEV Stat join(const Stat& x, const Stat& y, float c) {
  Stat z;
  z.m = max_nan(x.m, y.m);
  const float off = z.m == -INFINITY ? 0.f : z.m;
  z.s = x.s * ex2((x.m - off) * c) + y.s * ex2((y.m - off) * c);
  return z;
}

// ... of all the lanes of a warp: one maximum, one rescaling each
PE_DEV Stat warp_join(Stat x, float c) {
  float m = x.m;
#pragma unroll
  for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return Stat{m, warp_sum(x.s * ex2((x.m - (m == -INFINITY ? 0.f : m)) * c))};
}

// log2(e) / T rounded once (a division and a correction by its remainder)
PE_DEV float scale_of(float temp) {
  const float hi = 1.44269502162933349609375f, lo = 1.925963033500011e-8f;  // log2(e)
  const float q = hi / temp;
  return q + (fmaf(-q, temp, hi) + lo) / temp;
}

// Largest element of a 16-byte vector, NaN if it holds one.
PE_DEV uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <typename T>
PE_DEV float vec_max(const uint4& u);
template <>
PE_DEV float vec_max<float>(const uint4& u) {
  return max_nan(max_nan(__uint_as_float(u.x), __uint_as_float(u.y)),
                 max_nan(__uint_as_float(u.z), __uint_as_float(u.w)));
}
template <>
PE_DEV float vec_max<bf16>(const uint4& u) {
  const uint32_t p = max_nan_bf16x2(max_nan_bf16x2(u.x, u.y), max_nan_bf16x2(u.z, u.w));
  return max_nan(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 6) sampled_row_kernel(const VerifyArgs a) {
  constexpr int kVec = 16 / sizeof(T);
  __shared__ Stat st_sh[kThreads / 32];
  __shared__ unsigned long long key_sh[kThreads / 32];
  __shared__ float temp_sh;
  // (in this order: when the request kernel starts, what came before this one is done, and
  // the inputs may be read)
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x / a.splits, sp = blockIdx.x - row * a.splits;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x == 0) {  // only the request kernel, after this one, uses these
    if (tid == 0) *a.status = 0u;
    for (int r = tid; r < a.B; r += kThreads) a.done[r] = 0u;
  }
  const int c0 = sp * a.chunk, c1 = min(a.V, c0 + a.chunk);
  const T* base = static_cast<const T*>(a.logits) + static_cast<size_t>(row) * a.V;
  // scalar head up to the first 16-byte boundary, vectors, scalar tail
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(base + c0);
  const int head = min(static_cast<int>(((16u - (a0 & 15u)) & 15u) / sizeof(T)), c1 - c0);
  const int v0 = c0 + head, nvec = (c1 - v0) / kVec, t0 = v0 + nvec * kVec;
  const uint4* vp = reinterpret_cast<const uint4*>(base + v0);
  const uint4 none = sizeof(T) == 2 ? make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u)
                                    : make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
  // the first vectors are on their way while the row's request is looked up
  uint4 u[kUnroll];
#pragma unroll
  for (int x = 0; x < kUnroll; ++x)
    u[x] = tid + x * kThreads < nvec ? ld_stream16(vp + tid + x * kThreads) : none;
  if (warp == 0) {
    const int r = request_of(a, row, lane);
    if (lane == 0) temp_sh = r < 0 ? -1.f : temperature_of(given_temperature(a, r));
  }
  __syncthreads();
  const float temp = temp_sh;
  if (temp < 0.f) return;
  if (temp == 0.f) {
    // the first vector that holds this thread's greatest value stays in registers (a NaN
    // counts as the greatest); its lowest index with the value is found at the end
    unsigned long long k = 0ull;
    if (tid < head) k = argmax_key(Elem<T>::to_f(base[c0 + tid]), static_cast<uint32_t>(c0 + tid));
    float best = -INFINITY;
    int bj = -1;
    uint4 bv = none;
    for (int j = tid; j < nvec; j += kUnroll * kThreads) {
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) {
        const float m = vec_max<T>(u[x]);
        const int jx = j + x * kThreads, jn = jx + kUnroll * kThreads;
        if (jx < nvec && (bj < 0 || (!(m <= best) && best == best))) {
          best = m;
          bj = jx;
          bv = u[x];
        }
        if (jn < nvec) u[x] = ld_stream16(vp + jn);
      }
    }
    if (bj >= 0) {
      float f[kVec];
      unpack16<T>(bv, f);
      int e = kVec - 1;
#pragma unroll
      for (int i = kVec - 1; i >= 0; --i)
        if (best != best ? f[i] != f[i] : f[i] == best) e = i;
      k = max(k, argmax_key(best, static_cast<uint32_t>(v0 + bj * kVec + e)));
    }
    if (t0 + tid < c1)
      k = max(k, argmax_key(Elem<T>::to_f(base[t0 + tid]), static_cast<uint32_t>(t0 + tid)));
    k = warp_max_u64(k);
    if (lane == 0) key_sh[warp] = k;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kThreads / 32; ++w) k = max(k, key_sh[w]);
      a.rows[static_cast<size_t>(row) * a.splits + sp] = k;
    }
    return;
  }
  const float c = scale_of(temp);
  const uint64_t c2 = pack_f32x2(c, c);
  Stat st{-INFINITY, 0.f};
  if (tid < head) st = join(st, Stat{Elem<T>::to_f(base[c0 + tid]), 1.f}, c);
  if (t0 + tid < c1) st = join(st, Stat{Elem<T>::to_f(base[t0 + tid]), 1.f}, c);
  for (int j = tid; j < nvec; j += kUnroll * kThreads) {
    // one maximum and one rescaling for the kUnroll vectors
    float m = st.m;
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) m = max_nan(m, vec_max<T>(u[x]));
    const float off = m == -INFINITY ? 0.f : m;
    st.s *= ex2((st.m - off) * c);
    st.m = m;
    const int jn = j + kUnroll * kThreads;
    const uint64_t off2 = pack_f32x2(-off, -off);
    uint64_t s[2] = {0ull, 0ull};
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      float f[kVec];
      unpack16<T>(u[x], f);
      if (jn + x * kThreads < nvec)
        u[x] = ld_stream16(vp + jn + x * kThreads);
      else
        u[x] = none;
#pragma unroll
      for (int e = 0; e < kVec; e += 2) {
        float p, q;
        unpack_f32x2(mul_f32x2(add_f32x2(pack_f32x2(f[e], f[e + 1]), off2), c2), p, q);
        s[e / 2 & 1] = add_f32x2(s[e / 2 & 1], pack_f32x2(ex2(p), ex2(q)));
      }
    }
    float s0, s1;
    unpack_f32x2(add_f32x2(s[0], s[1]), s0, s1);
    st.s += s0 + s1;
  }
  st = warp_join(st, c);
  if (lane == 0) st_sh[warp] = st;
  __syncthreads();
  if (warp == 0) {
    st = warp_join(lane < kThreads / 32 ? st_sh[lane] : Stat{-INFINITY, 0.f}, c);
    if (lane == 0)
      a.rows[static_cast<size_t>(row) * a.splits + sp] =
          (static_cast<uint64_t>(__float_as_uint(st.m)) << 32) | __float_as_uint(st.s);
  }
}

// order of a score, larger first; -inf and NaN never win (key 0)
PE_DEV unsigned long long score_order(double x) {
  if (!(x > -INFINITY)) return 0ull;
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x + 0.0));
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

PE_DEV void warp_best(unsigned long long& k, int& v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const unsigned long long k2 = __shfl_xor_sync(0xffffffffu, k, o);
    const int v2 = __shfl_xor_sync(0xffffffffu, v, o);
    if (k2 > k || (k2 == k && v2 < v)) {
      k = k2;
      v = v2;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sampled_request_kernel(const VerifyArgs a) {
  constexpr int kW = kThreads / 32;
  __shared__ int bad_sh, last_sh;
  __shared__ uint32_t st_sh;
  __shared__ int pick_sh[kW];
  __shared__ float max_sh[kW];
  __shared__ float top_sh[kW];
  __shared__ unsigned long long key_sh[kW];
  __shared__ int idx_sh[kW];
  pdl_trigger();
  const int r = blockIdx.x / a.rsplits, sp = blockIdx.x - r * a.rsplits;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // The inputs are read while the row kernel ends (from L2: this kernel has waited for
  // nothing yet): the request, and of the row that this warp looks at first the draft, its
  // logit and its number (8 fp32 rows 11.4 -> 10.8 us).
  const RowRange x = row_range(__ldcg(a.qsl + r), __ldcg(a.qsl + r + 1), r, a.T);
  const int n = x.q1 - x.q0;
  const float t0 = given_temperature(a, r);
  const float temp = temperature_of(t0);
  struct Draft {
    int v;       // the draft after the row, -1: none
    float l, u;  // its logit in the row and its number
  };
  auto draft_of = [&](int j) {
    Draft d{-1, -INFINITY, 0.f};
    const int64_t row = x.q0 + j;
    if (j + 1 < n) {
      d.v = __ldcg(a.tok + row + 1);
      if (temp != 0.f) {
        d.u = __ldcg(a.u + row + 1);
        if (d.v >= 0 && d.v < a.V) d.l = Elem<T>::to_f(__ldcg(static_cast<const T*>(a.logits) + row * a.V + d.v));
      }
    }
    return d;
  };
  const Draft first = draft_of(warp);
  pdl_wait();
  if (temp == 0.f && sp > 0) return;  // a greedy request has no race
  uint32_t st = x.bad ? PE_ST_ROWS_RANGE : 0u;
  if (!(t0 >= 0.f)) st |= PE_ST_SAMPLING;
  if (tid == 0) {
    bad_sh = n;
    st_sh = 0u;
    if (sp == 0 && n > 0 && a.p_draft) a.p_draft[x.q0] = 1.f;
  }
  __syncthreads();
  int acc = 0, pick_acc = -1;
  float max_acc = 0.f;
  bool found = false;
  // One warp per row, in order: the row's statistics (or key), then the draft after
  // it.  The first CTA goes through all rows (p_draft), the others stop behind the
  // first rejection.
  const float c = temp == 0.f ? 1.f : scale_of(temp);
  const size_t rs = static_cast<size_t>(x.q0) * a.splits;
  auto row_stat = [&](int j) {
    Stat s{-INFINITY, 0.f};
    for (int i = lane; i < a.splits; i += 32) {
      const uint64_t w = a.rows[rs + static_cast<size_t>(j) * a.splits + i];
      s = join(s, Stat{__uint_as_float(static_cast<uint32_t>(w >> 32)),
                       __uint_as_float(static_cast<uint32_t>(w))}, c);
    }
    return warp_join(s, c);
  };
  auto row_pick = [&](int j) {
    unsigned long long k = 0ull;
    for (int i = lane; i < a.splits; i += 32)
      k = max(k, static_cast<unsigned long long>(a.rows[rs + static_cast<size_t>(j) * a.splits + i]));
    return static_cast<int>(~static_cast<uint32_t>(warp_max_u64(k)));
  };
  for (int j0 = 0; j0 < n; j0 += kW) {
    const int j = j0 + warp;
    int rejected = 0;
    if (j < n) {
      const int64_t row = x.q0 + j;
      const bool draft = j + 1 < n;
      const Draft d = j0 == 0 ? first : draft_of(j);
      const int v = d.v;
      const bool in = v >= 0 && v < a.V;
      float p = 0.f, top = 0.f;
      int pick = -1;
      if (temp == 0.f) {
        pick = row_pick(j);
        p = in && pick == v ? 1.f : 0.f;
      } else {
        const Stat s = row_stat(j);
        top = s.m;
        pick = fabsf(s.m) < INFINITY ? 0 : -1;  // whether the row has a distribution
        if (pick == 0) p = fminf(ex2((d.l - s.m) * c) / s.s, 1.f);
        rejected = !(d.u < p);
      }
      if (temp == 0.f) rejected = p == 0.f;
      rejected &= draft;
      if (draft && !in) st |= PE_ST_TOKEN_RANGE;
      if (lane == 0) {
        if (draft && sp == 0 && a.p_draft) a.p_draft[row + 1] = p;
        if (rejected) atomicMin(&bad_sh, j);
        pick_sh[warp] = pick;
        max_sh[warp] = top;
      }
    }
    // the first rejection (or the last row) decides what the next token comes from
    const bool any = __syncthreads_or(rejected);
    if (!found && (any || j0 + kW >= n)) {
      found = true;
      acc = min(bad_sh, n - 1);
      pick_acc = pick_sh[acc - j0];
      max_acc = max_sh[acc - j0];
    }
    __syncthreads();
    if (found && sp > 0) break;
  }
  const int64_t row = x.q0 + acc;
  int bonus = temp == 0.f ? pick_acc : -1;
  const bool race = n > 0 && temp != 0.f && pick_acc == 0;
  if (n > 0 && temp != 0.f && !race) st |= PE_ST_SAMPLING;
  if (sp == 0 && st) atomicOr(&st_sh, st);
  unsigned long long best = 0ull;
  int bi = 0x7fffffff;
  if (race) {
    const int skip = acc + 1 < n ? a.tok[row + 1] : -1;
    const T* lp = static_cast<const T*>(a.logits) + row * a.V;
    const float* gp = a.gumbel + static_cast<int64_t>(r) * a.V;
    const int c0 = sp * a.rchunk, c1 = min(a.V, c0 + a.rchunk);
    const float it = (1.f / temp);
    float bs = -INFINITY;
    // The score counts from the row's largest logit: the difference is exact near it, and
    // no quotient passes fp32's range upwards.  A logit of -inf gives -inf, or NaN with
    // infinite noise: neither is greater than anything.
    const uint64_t it2 = pack_f32x2(it, it), off2 = pack_f32x2(-max_acc, -max_acc);
    auto scores = [&](const float* l, const float* g, int v, float* x) {  // of kRace tokens from v
#pragma unroll
      for (int e = 0; e < kRace; e += 2)
        unpack_f32x2(fma_f32x2(add_f32x2(pack_f32x2(l[e], l[e + 1]), off2), it2, pack_f32x2(g[e], g[e + 1])),
                     x[e], x[e + 1]);
      if (static_cast<unsigned>(skip - v) < kRace) {
#pragma unroll
        for (int e = 0; e < kRace; ++e)
          if (v + e == skip) x[e] = -INFINITY;
      }
    };
    constexpr int kVecs = sizeof(T) == 2 ? 1 : 2;  // 16-byte vectors of kRace logits
    constexpr int kStep = kThreads * kRace;
    int v = c0 + tid * kRace;
    if (a.vec) {
      for (; v + kRace <= c1; v += kRaceRounds * kStep) {
        // all the rounds' loads first
        uint4 lv[kRaceRounds][kVecs], gv[kRaceRounds][2];
#pragma unroll
        for (int x = 0; x < kRaceRounds; ++x)
          if (v + x * kStep + kRace <= c1) {
#pragma unroll
            for (int y = 0; y < kVecs; ++y)
              lv[x][y] = *reinterpret_cast<const uint4*>(lp + v + x * kStep + y * (kRace / kVecs));
            gv[x][0] = ld_stream16(gp + v + x * kStep);
            gv[x][1] = ld_stream16(gp + v + x * kStep + 4);
          }
#pragma unroll
        for (int x = 0; x < kRaceRounds; ++x)
          if (v + x * kStep + kRace <= c1) {
            float l[kRace], g[kRace];
#pragma unroll
            for (int y = 0; y < kVecs; ++y) unpack16<T>(lv[x][y], l + y * (kRace / kVecs));
            unpack16<float>(gv[x][0], g);
            unpack16<float>(gv[x][1], g + 4);
            float sc[kRace];
            scores(l, g, v + x * kStep, sc);
            float m = sc[0];
#pragma unroll
            for (int e = 1; e < kRace; ++e) m = fmaxf(m, sc[e]);
            if (m > bs) {
              bs = m;
              bi = v + x * kStep;  // the first vector with the best score
            }
          }
      }
    } else {
      for (v = c0 + tid; v < c1; v += kRace * kThreads) {
        float l[kRace], g[kRace];
#pragma unroll
        for (int e = 0; e < kRace; ++e) {
          const int w = v + e * kThreads;
          l[e] = w < c1 ? Elem<T>::to_f(lp[w]) : -INFINITY;
          g[e] = w < c1 ? gp[w] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < kRace; ++e) {
          const int w = v + e * kThreads;
          const float x = w == skip ? -INFINITY : fmaf(l[e] - max_acc, it, g[e]);
          if (x > bs) {
            bs = x;
            bi = w;
          }
        }
      }
    }
    // The threads whose best is within reach of the CTA's (a score's rounding is 2^-23 of
    // its two terms; noise past 128 is infinite) compare in 64 bits: doubles are slow here,
    // and by then it is one or two of the 256.
    float top = warp_max(bs);
    if (lane == 0) top_sh[warp] = top;
    __syncthreads();
    top = top_sh[0];
#pragma unroll
    for (int w = 1; w < kW; ++w) top = fmaxf(top, top_sh[w]);
    if (bs > -INFINITY && (bs == top || bs >= top - 1e-6f * (fabsf(top) + fabsf(bs) + 128.f))) {
      float l[kRace], g[kRace], sc[kRace];
      float bl = 0.f, bg = 0.f;
      if (a.vec) {  // the first token of the vector with that score
#pragma unroll
        for (int e = 0; e < kRace; ++e) {
          l[e] = Elem<T>::to_f(lp[bi + e]);
          g[e] = gp[bi + e];
        }
        scores(l, g, bi, sc);
        int first = 0;
#pragma unroll
        for (int e = kRace - 1; e >= 0; --e)
          if (sc[e] == bs) {
            first = e;
            bl = l[e];
            bg = g[e];
          }
        bi += first;
      } else {
        bl = Elem<T>::to_f(lp[bi]);
        bg = gp[bi];
      }
      best = score_order((static_cast<double>(bl) - static_cast<double>(max_acc)) / static_cast<double>(temp) + bg);
    } else {
      bi = 0x7fffffff;
    }
    warp_best(best, bi);
    if (lane == 0) {
      key_sh[warp] = best;
      idx_sh[warp] = bi;
    }
    __syncthreads();
    if (warp == 0) {
      best = lane < kW ? key_sh[lane] : 0ull;
      bi = lane < kW ? idx_sh[lane] : 0x7fffffff;
      warp_best(best, bi);
    }
  }
  __syncthreads();
  if (tid == 0) {
    if (st_sh) set_status(a.status, st_sh);
    last_sh = 1;
    if (race) {
      a.best[static_cast<size_t>(r) * a.rsplits + sp] =
          make_ulonglong2(best, static_cast<unsigned long long>(bi));
      __threadfence();
      last_sh = atomicAdd(&a.done[r], 1u) == static_cast<uint32_t>(a.rsplits) - 1u;
    } else if (sp > 0) {
      last_sh = 0;
    }
  }
  __syncthreads();
  if (!last_sh || warp != 0) return;
  if (race) {
    __threadfence();
    best = 0ull;
    bi = 0x7fffffff;
    for (int i = lane; i < a.rsplits; i += 32) {
      const volatile ulonglong2* e = a.best + static_cast<size_t>(r) * a.rsplits + i;
      const unsigned long long k = e->x;
      const int v = static_cast<int>(e->y);
      if (k > best || (k == best && v < bi)) {
        best = k;
        bi = v;
      }
    }
    warp_best(best, bi);
    bonus = best ? bi : -1;
  }
  if (lane == 0) {
    a.accepted[r] = acc;
    a.bonus[r] = bonus;
  }
}

size_t al256(size_t x) { return (x + 255) / 256 * 256; }

// Chunks of a row: about one wave of CTAs (six per SM) over the batch, at least one
// 16-byte vector per thread, at most 64 KB.  Chunks of the race: about four CTAs
// per SM, whole trips of the loop (64 requests: 59.5 us the call, 62.2 with a part of a trip
// left over), at least one round per thread.
void plan(VerifyArgs& a, int esize, int num_sms) {
  const int vec = 16 / esize;
  const long long total = static_cast<long long>(a.T) * a.V;
  long long chunk = (total + 6LL * num_sms - 1) / (6LL * num_sms);
  chunk = std::max<long long>(chunk, static_cast<long long>(kThreads) * vec);
  chunk = std::min<long long>(chunk, kMaxChunkBytes / esize);
  chunk = (chunk + vec - 1) / vec * vec;
  a.chunk = static_cast<int>(chunk);
  a.splits = static_cast<int>((a.V + chunk - 1) / chunk);
  const long long noise = static_cast<long long>(a.B) * a.V;
  chunk = std::max<long long>((noise + 4LL * num_sms - 1) / (4LL * num_sms), kThreads * kRace);
  constexpr long long kTrip = kThreads * kRace * kRaceRounds;
  chunk = std::max<long long>((chunk + kTrip / 2) / kTrip * kTrip, kThreads * kRace);
  a.rchunk = static_cast<int>(std::min<long long>(chunk, 0x7ffffff8));
  a.rsplits = static_cast<int>((a.V + chunk - 1) / chunk);
}

// the most chunks a row (one fp32 vector per thread) and a race can have
size_t max_splits(int V) { return (static_cast<size_t>(V) + kThreads * 4 - 1) / (kThreads * 4); }
size_t max_rsplits(int V) { return (static_cast<size_t>(V) + kThreads * kRace - 1) / (kThreads * kRace); }
constexpr int kWsHeader = 256;

}  // namespace
}  // namespace pe

using namespace pe;

extern "C" size_t pe_verify_sampled_workspace_bytes(int max_batch, int max_rows_in, int vocab) {
  if (max_batch < 0 || max_rows_in < 0 || vocab < 1) return 0;
  return kWsHeader + al256(max_rows_in * max_splits(vocab) * sizeof(uint64_t)) +
         al256(max_batch * sizeof(uint32_t)) + max_batch * max_rsplits(vocab) * sizeof(ulonglong2);
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
  if (B > 65535 || vocab > 1 << 30) return PE_ERR_UNSUPPORTED;
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
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return PE_ERR_CUDA;
  VerifyArgs a = {};
  a.B = B;
  a.T = T_in;
  a.V = vocab;
  a.qsl = qsl;
  a.tok = tok;
  a.logits = logits;
  a.temperature = temperature;
  a.u = u;
  a.gumbel = gumbel;
  a.accepted = accepted;
  a.bonus = bonus;
  a.p_draft = p_draft;
  plan(a, esize, sms);
  a.vec = vocab % 8 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0 &&
          reinterpret_cast<uintptr_t>(gumbel) % 16 == 0;
  if (static_cast<long long>(T_in) * a.splits > 0x7fffffffLL ||
      static_cast<long long>(B) * a.rsplits > 0x7fffffffLL)
    return PE_ERR_UNSUPPORTED;
  char* w = static_cast<char*>(ws);
  a.status = reinterpret_cast<uint32_t*>(w);
  w += kWsHeader;
  a.rows = reinterpret_cast<uint64_t*>(w);
  w += al256(T_in * max_splits(vocab) * sizeof(uint64_t));
  a.done = reinterpret_cast<uint32_t*>(w);
  w += al256(B * sizeof(uint32_t));
  a.best = reinterpret_cast<ulonglong2*>(w);
  const bool f32 = dtype == PE_DTYPE_F32;
  if (T_in > 0) {
    if (launch_chained(f32 ? sampled_row_kernel<float> : sampled_row_kernel<bf16>,
                       dim3(static_cast<unsigned>(T_in) * a.splits), dim3(kThreads), 0, st, a) != cudaSuccess)
      return PE_ERR_CUDA;
  } else if (cudaMemsetAsync(ws, 0, sizeof(uint32_t), st) != cudaSuccess) {
    return PE_ERR_CUDA;
  }
  return launch_chained(f32 ? sampled_request_kernel<float> : sampled_request_kernel<bf16>,
                        dim3(static_cast<unsigned>(B) * a.rsplits), dim3(kThreads), 0, st, a) == cudaSuccess
             ? PE_OK
             : PE_ERR_CUDA;
}
