// The target's token after each row: temperature, top-k, top-p, min-p, from given noise
// (pe_sample).
//
// The kept tokens are the first ones of one order (logit descending, index ascending), as many
// as all three settings allow, so a row's answer needs the place of the cut in that order and
// then the best of (l - max) / T + g over the tokens before it.  Nothing is sorted as a whole.
//
//   row kernel   CTA (row, part) streams its part of the logits once: the largest logit, the
//                sum of weights (top-p), the first largest token (greedy) or the best score
//                (nothing is cut: the noise is streamed along).  For rows with a cut it also
//                leaves the largest logit of each group of some hundred tokens.
//   cut kernel   a CTA per row joins the parts.  For a row with a cut:
//                  - a bound from below for it.  The groups' largest logits are tokens of the
//                    row, so the value at which k of them (for top-p: enough of them to weigh
//                    p of the whole) are reached cannot lie above the cut;
//                  - the tokens from the bound on, read again from the few groups that have
//                    one: rank and weight before each by comparing all pairs, the cut, the
//                    best score.
//   wide kernel  takes the rows for which that does not do (flat rows that keep thousands of
//                tokens, a large k, many equal logits), a cluster of CTAs a row with a slice
//                each in shared memory: histograms of counts and weights over the distance from the
//                largest logit, finer ones inside the bin of the cut, then a race over the
//                slices.  Weights are 31-bit integers there: their sums do not depend on the
//                order of the atomics.
//
// The first kernel is bound by the logits' bytes.  (Every row by a cluster with the row in
// shared memory: 512 bf16 rows of 201,088 with top-k 162 us; the barriers of a row are waited
// for with its 400 KB held.)
#include <algorithm>
#include <atomic>
#include <cmath>

#include "pe_paged.h"
#include "pe_sampling.cuh"

namespace pe {
namespace {

constexpr int kThreads = 256;         // row kernel
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;            // 16-byte loads in flight per thread
constexpr int kRaceUnroll = 2;        // ... where the noise is streamed too
constexpr int kMaxPartBytes = 65536;  // of a row, per CTA
constexpr int kGroups = 4096;         // of a row, at most
constexpr int kBins = 256;
constexpr int kList = 512;            // candidates of a row whose pairs are compared
constexpr int kGroupList = 1024;      // groups that are read again

constexpr int kWideThreads = 512;     // wide kernel
constexpr int kWideWarps = kWideThreads / 32;
constexpr int kCluster = 8;

// What a CTA of the row kernel leaves of its part.
struct __align__(16) Part {
  float m;        // largest logit (NaN if there is one)
  float s;        // sum of weights relative to it
  float x, g;     // of the best score: logit and noise
  int idx;        // ... and token, -1: there is none
  int pad;
  unsigned long long key;  // greedy: argmax_key of the first largest logit
};

struct Settings;

struct SampleArgs {
  int B, T, V;
  const int32_t* qsl;
  const void* logits;
  int64_t ld;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* gumbel;
  int64_t ld_g;
  int32_t* token;
  uint32_t* status;
  int part, parts;   // 16-byte vectors of a part, parts of a row
  int gshift;        // threads of a group: 1 << gshift
  Part* stat;        // [T][parts]
  float* top;        // [T][parts][kThreads >> gshift]
  Settings* set;  // [T] of each row
  uint32_t* todo_n;  // rows for the wide kernel
  int32_t* todo;     // [T]
  int resident;      // the wide kernel's slices fit in shared memory
};

struct Settings {
  float temp, p, mp;  // temperature (negative: a row of no request); top-p, 1: off; min-p, 0: off
  int k;              // 0: off
};
PE_DEV Settings settings_of(const SampleArgs& a, int r, uint32_t& status) {
  Settings s;
  const float t = a.temperature ? a.temperature[r] : 1.f;
  const int k = a.top_k ? a.top_k[r] : 0;
  const float p = a.top_p ? a.top_p[r] : 1.f, mp = a.min_p ? a.min_p[r] : 0.f;
  if (!(t >= 0.f) || p != p || mp != mp) status |= PE_ST_SAMPLING;
  s.temp = temperature_of(t);
  s.k = k <= 0 || k >= a.V ? 0 : k;
  s.p = p < 1.f ? p : 1.f;     // (NaN: 1)
  s.mp = mp > 0.f ? mp : 0.f;  // (NaN: 0)
  return s;
}

// A row in 16-byte vectors on the grid of the addresses: vector v holds the tokens
// v * kVec - shift and on, those outside the row as -inf.
template <typename T>
struct Row {
  static constexpr int kVec = 16 / sizeof(T);
  const T* row;
  int V, shift;
  PE_DEV Row(const SampleArgs& a, int r) {
    row = static_cast<const T*>(a.logits) + r * a.ld;
    V = a.V;
    shift = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
  }
  PE_DEV int vectors() const { return (V + shift + kVec - 1) / kVec; }
  PE_DEV int token(int v) const { return v * kVec - shift; }
  PE_DEV uint4 load(int v) const {
    const int e = token(v);
    if (e >= 0 && e + kVec <= V) return ld_stream16(row + e);
    float f[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[i] = e + i >= 0 && e + i < V ? Elem<T>::to_f(row[e + i]) : -INFINITY;
    return pack16<T>(f);
  }
};
template <typename T>
PE_DEV uint4 no_tokens() {
  return sizeof(T) == 2 ? make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u)
                        : make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
}

// The noise of a row beside a vector of its logits; zeros outside the row.
template <typename T>
struct Noise {
  static constexpr int kVec = 16 / sizeof(T);
  const float* g;
  bool wide;  // vectors of noise lie on the 16-byte grid too
  PE_DEV Noise(const SampleArgs& a, int r, int shift) {
    g = a.gumbel + r * a.ld_g;
    wide = !((reinterpret_cast<uintptr_t>(g) - shift * 4u) & 15u);
  }
  PE_DEV void load(int t0, int V, float* x) const {
    if (wide && t0 >= 0 && t0 + kVec <= V) {
#pragma unroll
      for (int e = 0; e < kVec; e += 4) unpack16<float>(ld_stream16(g + t0 + e), x + e);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) x[e] = t0 + e >= 0 && t0 + e < V ? g[t0 + e] : 0.f;
    }
  }
};

PE_DEV unsigned long long exact_score(float x, float g, float M, float temp) {
  return score_order((static_cast<double>(x) - static_cast<double>(M)) / static_cast<double>(temp) + g);
}

// The logit of an order (argmax_order)
PE_DEV float logit_of(uint32_t order) {
  return __uint_as_float(order & 0x80000000u ? order & 0x7fffffffu : ~order);
}

// Best (order, index) of the CTA; all threads get it.
template <int W>
PE_DEV void cta_best(unsigned long long& k, int& i, unsigned long long* ks, int* is) {
  warp_best(k, i);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    ks[threadIdx.x >> 5] = k;
    is[threadIdx.x >> 5] = i;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  k = lane < W ? ks[lane] : 0ull;
  i = lane < W ? is[lane] : 0x7fffffff;
  warp_best(k, i);
}
template <int W>
PE_DEV float cta_max(float v, float* warps) {  // NaN if there is one
#pragma unroll
  for (int o = 16; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
  __syncthreads();
  v = warps[0];
  for (int w = 1; w < W; ++w) v = max_nan(v, warps[w]);
  return v;
}
// Sum over the CTA, in a fixed order; all threads get it.
template <int W>
PE_DEV double cta_sum(double v, double* warps) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.;
  for (int w = 0; w < W; ++w) s += warps[w];
  return s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) sample_row_kernel(const SampleArgs a) {
  constexpr int kVec = 16 / sizeof(T);
  __shared__ float warp_m[kWarps];
  __shared__ double warp_d[kWarps];
  __shared__ unsigned long long warp_k[kWarps];
  __shared__ int warp_i[kWarps];
  __shared__ Settings set_sh;
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x / a.parts, part = blockIdx.x - row * a.parts;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Row<T> s(a, row);
  const int v0 = part * a.part, n = min(a.part, s.vectors() - v0);  // (n <= 0: nothing is left for this part)
  // the first vectors are on their way while the row's request is looked up
  uint4 u[kUnroll];
#pragma unroll
  for (int x = 0; x < kUnroll; ++x) u[x] = tid + x * kThreads < n ? s.load(v0 + tid + x * kThreads) : no_tokens<T>();
  if (warp == 0) {
    const int r = request_of(a.qsl, a.B, row, lane);
    if (lane == 0) {
      uint32_t status = 0;
      Settings x{-1.f, 1.f, 0.f, 0};
      if (r >= 0) {
        x = settings_of(a, r, status);
        if (request_rows(a.qsl, r, a.T).bad) status |= PE_ST_ROWS_RANGE;
      }
      set_sh = x;
      if (part == 0) {
        a.set[row] = x;
        if (status) set_status(a.status, status);
        if (row == 0) *a.todo_n = 0u;
      }
    }
  }
  __syncthreads();
  const Settings st = set_sh;
  if (st.temp < 0.f) return;
  Part out{-INFINITY, 0.f, 0.f, 0.f, -1, 0, 0ull};
  const bool free = st.k == 0 && st.p >= 1.f && st.mp == 0.f;
  float m = -INFINITY;
  if (st.temp == 0.f) {
    // the first vector that holds this thread's greatest value stays in registers (a NaN
    // counts as the greatest); its lowest index with the value is found at the end
    int bj = -1;
    uint4 bv = no_tokens<T>();
    for (int j = tid; j < n; j += kUnroll * kThreads) {
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) {
        const float vm = vec_max<T>(u[x]);
        const int jx = j + x * kThreads, jn = jx + kUnroll * kThreads;
        if (jx < n && (bj < 0 || (!(vm <= m) && m == m))) {
          m = vm;
          bj = jx;
          bv = u[x];
        }
        if (jn < n) u[x] = s.load(v0 + jn);
      }
    }
    unsigned long long k = 0ull;
    if (bj >= 0) {
      float f[kVec];
      unpack16<T>(bv, f);
      const int t0 = s.token(v0 + bj);
#pragma unroll
      for (int e = kVec - 1; e >= 0; --e)
        if (t0 + e >= 0 && t0 + e < a.V && (m != m ? f[e] != f[e] : f[e] == m))
          k = argmax_key(m, static_cast<uint32_t>(t0 + e));
    }
    k = warp_max_u64(k);
    if (lane == 0) warp_k[warp] = k;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) k = max(k, warp_k[w]);
    out.key = k;
  } else if (free) {
    // (l - m) / T + g with the thread's largest logit so far: exact near it, and no quotient
    // passes fp32's range upwards
    const Noise<T> noise(a, row, s.shift);
    const float it = 1.f / st.temp;
    float bs = -INFINITY;
    int bv = -1;
    for (int j = tid; j < n; j += kRaceUnroll * kThreads) {
      if (j != tid) {
#pragma unroll
        for (int x = 0; x < kRaceUnroll; ++x)
          u[x] = j + x * kThreads < n ? s.load(v0 + j + x * kThreads) : no_tokens<T>();
      }
      float g[kRaceUnroll][kVec];
#pragma unroll
      for (int x = 0; x < kRaceUnroll; ++x)
        if (j + x * kThreads < n) noise.load(s.token(v0 + j + x * kThreads), a.V, g[x]);
      float mn = m;
#pragma unroll
      for (int x = 0; x < kRaceUnroll; ++x) mn = max_nan(mn, vec_max<T>(u[x]));
      const float off = mn == -INFINITY ? 0.f : mn;
      if (mn > m && bs < INFINITY) bs = fmaf(m - mn, it, bs);
      m = mn;
#pragma unroll
      for (int x = 0; x < kRaceUnroll; ++x) {
        if (j + x * kThreads >= n) continue;
        float f[kVec], best = -INFINITY;
        unpack16<T>(u[x], f);
#pragma unroll
        for (int e = 0; e < kVec; ++e) best = fmaxf(best, fmaf(f[e] - off, it, g[x][e]));
        if (best > bs || bv < 0) {
          bs = fmaxf(bs, best);
          bv = j + x * kThreads;
        }
      }
    }
    out.m = cta_max<kWarps>(m, warp_m);
    // The threads whose best is within reach of the CTA's (a score's rounding is 2^-23 of its
    // terms; noise past 128 is infinite) compare in 64 bits, token by token.
    const float far = m == out.m ? 0.f : (m - out.m) * it;
    if (bs < INFINITY) bs += far;
    float top = warp_max(bs);
    __syncthreads();
    if (lane == 0) warp_m[warp] = top;
    __syncthreads();
    top = warp_m[0];
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, warp_m[w]);
    unsigned long long k = 0ull;
    int bi = 0x7fffffff;
    float bx = 0.f, bg = 0.f;
    if (bv >= 0 && fabsf(out.m) < INFINITY &&
        (bs >= top || bs >= top - 1e-6f * (fabsf(top) + fabsf(bs) + fabsf(far) + 128.f))) {
      float f[kVec], g[kVec];
      unpack16<T>(s.load(v0 + bv), f);
      const int t0 = s.token(v0 + bv);
      noise.load(t0, a.V, g);
      for (int e = 0; e < kVec; ++e) {
        const unsigned long long o = f[e] == -INFINITY ? 0ull : exact_score(f[e], g[e], out.m, st.temp);
        if (o > k) {
          k = o;
          bi = t0 + e;
          bx = f[e];
          bg = g[e];
        }
      }
    }
    unsigned long long best = k;
    int winner = bi;
    cta_best<kWarps>(best, winner, warp_k, warp_i);
    out.idx = best ? winner : -1;
    // (its thread writes the part)
    if (best ? bi == winner : tid == 0) {
      out.x = bx;
      out.g = bg;
      a.stat[static_cast<size_t>(row) * a.parts + part] = out;
    }
  } else if (st.k > 0 || st.p >= 1.f) {
    for (int j = tid; j < n; j += kUnroll * kThreads) {
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) {
        m = max_nan(m, vec_max<T>(u[x]));
        const int jn = j + (x + kUnroll) * kThreads;
        u[x] = jn < n ? s.load(v0 + jn) : no_tokens<T>();
      }
    }
  } else {
    // sum of 2^((l - m) c), c = log2(e) / T: the difference is exact near the largest logit
    const float c = scale_of(st.temp);
    const uint64_t c2 = pack_f32x2(c, c);
    float sum = 0.f;
    for (int j = tid; j < n; j += kUnroll * kThreads) {
      // one maximum and one rescaling for the kUnroll vectors
      float mn = m;
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) mn = max_nan(mn, vec_max<T>(u[x]));
      const float off = mn == -INFINITY ? 0.f : mn;
      sum *= ex2((m - off) * c);
      m = mn;
      const uint64_t off2 = pack_f32x2(-off, -off);
      uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) {
        float f[kVec];
        unpack16<T>(u[x], f);
        const int jn = j + (x + kUnroll) * kThreads;
        u[x] = jn < n ? s.load(v0 + jn) : no_tokens<T>();
#pragma unroll
        for (int e = 0; e < kVec; e += 2) {
          float p, q;
          unpack_f32x2(mul_f32x2(add_f32x2(pack_f32x2(f[e], f[e + 1]), off2), c2), p, q);
          acc[e / 2 & 1] = add_f32x2(acc[e / 2 & 1], pack_f32x2(ex2(p), ex2(q)));
        }
      }
      float s0, s1;
      unpack_f32x2(add_f32x2(acc[0], acc[1]), s0, s1);
      sum += s0 + s1;
    }
    out.m = cta_max<kWarps>(m, warp_m);
    out.s = static_cast<float>(
        cta_sum<kWarps>(m > -INFINITY ? sum * ex2((m - out.m) * c) : 0.f, warp_d));
  }
  if (!free && st.temp != 0.f) {
    if (st.k > 0 || st.p >= 1.f) out.m = cta_max<kWarps>(m, warp_m);
    float t = m;
    for (int o = 1; o < 1 << a.gshift; o <<= 1) t = max_nan(t, __shfl_xor_sync(0xffffffffu, t, o));
    if ((lane & ((1 << a.gshift) - 1)) == 0)
      a.top[(static_cast<size_t>(row) * a.parts + part) * (kThreads >> a.gshift) + (tid >> a.gshift)] = t;
  }
  if ((!free || st.temp == 0.f) && tid == 0) a.stat[static_cast<size_t>(row) * a.parts + part] = out;
}

// Candidates of a row, all tokens that come before some place in its order, and what comes
// before them (weights 2^-40): which are kept, and the best score.
struct Cands {
  unsigned long long key[kList];  // argmax_key: larger comes first
  unsigned long long q[kList];    // weight
  float g[kList];
};
constexpr float kOne = 0x1p40f;

// Shared memory of the cut kernel.
struct __align__(16) CutShared {
  float m[kWarps];
  double d[kWarps];
  unsigned long long k[kWarps];
  int i[kWarps];
  int n, n_groups, enough;
  uint32_t bound;
  float top[kGroups];
  union {
    struct {
      uint32_t cnt[kBins], least[kBins];  // of the groups' largest logits; order of the least
      unsigned long long mass[kBins];
    } h;
    Cands c;
  };
  uint16_t group[kGroupList];
};

// The answer of a row from its parts.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) sample_cut_kernel(const SampleArgs a) {
  constexpr int kVec = 16 / sizeof(T);
  __shared__ CutShared sh;
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Settings st = a.set[row];
  if (st.temp < 0.f) return;
  const Part* stat = a.stat + static_cast<size_t>(row) * a.parts;
  auto answer = [&](unsigned long long k, int i) {
    cta_best<kWarps>(k, i, sh.k, sh.i);
    if (tid == 0) {
      a.token[row] = k ? i : -1;
      if (!k) set_status(a.status, PE_ST_SAMPLING);
    }
  };
  if (st.temp == 0.f) {
    unsigned long long k = 0ull;
    for (int i = tid; i < a.parts; i += kThreads) k = max(k, __ldcg(&stat[i].key));
    answer(k, static_cast<int>(~static_cast<uint32_t>(k)));
    return;
  }
  float M = -INFINITY;
  for (int i = tid; i < a.parts; i += kThreads) M = max_nan(M, __ldcg(&stat[i].m));
  M = cta_max<kWarps>(M, sh.m);
  if (!(fabsf(M) < INFINITY)) {  // no distribution
    answer(0ull, -1);
    return;
  }
  const bool cut_k = st.k > 0, cut_p = st.p < 1.f;
  if (!cut_k && !cut_p && st.mp == 0.f) {
    unsigned long long k = 0ull;
    int best = 0x7fffffff;
    for (int i = tid; i < a.parts; i += kThreads) {
      const int t = __ldcg(&stat[i].idx);
      const unsigned long long o = t < 0 ? 0ull : exact_score(__ldcg(&stat[i].x), __ldcg(&stat[i].g), M, st.temp);
      if (o > k || (o == k && t < best)) {
        k = o;
        best = t;
      }
    }
    answer(k, best);
    return;
  }
  const float c = scale_of(st.temp);
  double z = 0.;  // the weight of the whole row
  if (cut_p && !cut_k) {
    for (int i = tid; i < a.parts; i += kThreads) {
      const float m = __ldcg(&stat[i].m);
      if (m > -INFINITY) z += static_cast<double>(__ldcg(&stat[i].s) * ex2((m - M) * c));
    }
    z = cta_sum<kWarps>(z, sh.d);
  }
  // ---------------- a bound from below for the cut
  const int gpp = kThreads >> a.gshift, groups = a.parts * gpp;  // groups of a part, of the row
  const float* top = a.top + static_cast<size_t>(row) * groups;
  float lo = INFINITY;
  for (int i = tid; i < groups; i += kThreads) {
    const float t = __ldcg(top + i);
    sh.top[i] = t;
    if (t > -INFINITY) lo = fminf(lo, t);
  }
  for (int b = tid; b < kBins; b += kThreads) {
    sh.h.cnt[b] = 0;
    sh.h.least[b] = 0xffffffffu;
    sh.h.mass[b] = 0;
  }
  if (tid == 0) {
    sh.n = sh.n_groups = 0;
    sh.enough = 0;
  }
  lo = -cta_max<kWarps>(-lo, sh.m);
  float bound = -INFINITY;
  if (cut_k || cut_p) {
    // bins of the range that the groups' largest logits span
    const float span = M - lo;
    const float scale = span > 0.f && span < INFINITY ? fminf(kBins / span, 1e30f) : 0.f;
    for (int i = tid; i < groups; i += kThreads) {
      const float t = sh.top[i];
      if (t > -INFINITY) {
        const int b = min(kBins - 1, static_cast<int>((M - t) * scale));
        atomicAdd(&sh.h.cnt[b], 1u);
        atomicMin(&sh.h.least[b], argmax_order(t));
        if (!cut_k) atomicAdd(&sh.h.mass[b], static_cast<unsigned long long>(ex2((t - M) * c) * kOne));
      }
    }
    __syncthreads();
    if (warp == 0) {
      // The first bin with which there are k, or p of the weight; for want of the latter as many
      // as can be compared (their weight tells, below).
      constexpr int kPer = kBins / 32;
      double have[kPer], mine = 0.;
      uint32_t count = 0;
      const double need = cut_k ? static_cast<double>(st.k) : z * fmaxf(st.p, 0.f) * 1.000001 * kOne;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int b = lane * kPer + e;
        have[e] = cut_k ? static_cast<double>(sh.h.cnt[b]) : static_cast<double>(sh.h.mass[b]);
        mine += have[e];
        count += sh.h.cnt[b];
      }
      double before = mine;
      uint32_t n_before = count;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, before, o);
        const uint32_t n = __shfl_up_sync(0xffffffffu, n_before, o);
        if (lane >= o) {
          before += y;
          n_before += n;
        }
      }
      before -= mine;
      n_before -= count;
      int last = kBins, most = -1;  // the bin; the last one with few enough groups before its end
#pragma unroll
      for (int e = kPer - 1; e >= 0; --e) {
        double upto = before;
        uint32_t n = n_before;
        for (int f = 0; f <= e; ++f) {
          upto += have[f];
          n += sh.h.cnt[lane * kPer + f];
        }
        if (upto >= need) last = lane * kPer + e;
        if (n <= kList / 2 && most < 0) most = lane * kPer + e;
      }
      last = __reduce_min_sync(0xffffffffu, last);
      most = __reduce_max_sync(0xffffffffu, most);
      if (last == kBins && !cut_k) last = most;
      uint32_t o = 0xffffffffu;
      for (int e = 0; e < kPer; ++e)
        if (lane * kPer + e <= last) o = min(o, sh.h.least[lane * kPer + e]);
      o = __reduce_min_sync(0xffffffffu, o);
      if (lane == 0) {
        sh.bound = o;
        sh.enough = last < kBins && last >= 0 && o != 0xffffffffu;
      }
    }
    __syncthreads();
    if (sh.enough) bound = logit_of(sh.bound);
  } else if (tid == 0) {
    sh.enough = 1;  // min-p alone: the weights say it
  }
  __syncthreads();
  bool done = sh.enough;
  if (done) {
    // ---------------- the groups that have a token from the bound on, and those tokens
    const bool by_w = !cut_k && !cut_p;
    auto in = [&](float x) { return by_w ? x == M || ex2((x - M) * c) >= st.mp : x >= bound; };
    for (int i = tid; i < groups; i += kThreads)
      if (sh.top[i] > -INFINITY && in(sh.top[i])) {
        const int at = atomicAdd(&sh.n_groups, 1);
        if (at < kGroupList) sh.group[at] = static_cast<uint16_t>(i);
      }
    __syncthreads();
    const Row<T> s(a, row);
    const int nv = s.vectors(), n_groups = sh.n_groups;
    if (n_groups <= kGroupList) {
      // a group's vectors: of each trip over the part, as many as it has threads
      const int trips = (a.part + kThreads - 1) / kThreads, per = trips << a.gshift;
      for (int i = tid; i < n_groups * per; i += kThreads) {
        const int g = sh.group[i / per], j = i % per;
        const int at = (j >> a.gshift) * kThreads + ((g % gpp) << a.gshift) + (j & ((1 << a.gshift) - 1));
        const int v = g / gpp * a.part + at;
        if (at >= a.part || v >= nv) continue;
        const uint4 u = s.load(v);
        if (!in(vec_max<T>(u))) continue;
        float f[kVec];
        unpack16<T>(u, f);
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          if (f[e] > -INFINITY && in(f[e])) {
            const int at2 = atomicAdd(&sh.n, 1);
            if (at2 < kList) sh.c.key[at2] = argmax_key(f[e], static_cast<uint32_t>(s.token(v) + e));
          }
      }
    }
    __syncthreads();
    const int n = sh.n;
    done = n_groups <= kGroupList && n <= kList;
    if (done) {
      // ---------------- rank and weight before each
      constexpr int kPer = kList / kThreads;
      const float* noise = a.gumbel + row * a.ld_g;
      unsigned long long key[kPer], before[kPer];
      float g[kPer];
      int place[kPer];
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        const int i = tid + x * kThreads;
        key[x] = before[x] = 0ull;
        place[x] = 0;
        g[x] = 0.f;
        if (i < n) {
          key[x] = sh.c.key[i];
          g[x] = noise[~static_cast<uint32_t>(key[x])];
          sh.c.q[i] = static_cast<unsigned long long>(ex2((logit_of(static_cast<uint32_t>(key[x] >> 32)) - M) * c) * kOne);
        }
      }
      __syncthreads();
      if ((tid & ~31) < n) {
        for (int j = 0; j < n; ++j) {
          const unsigned long long kj = sh.c.key[j], qj = sh.c.q[j];
#pragma unroll
          for (int x = 0; x < kPer; ++x)
            if (kj > key[x]) {
              ++place[x];
              before[x] += qj;
            }
        }
      }
      double sum = z * kOne;  // what top-p is a share of
      if (cut_p) {
        double mine = 0.;
#pragma unroll
        for (int x = 0; x < kPer; ++x)
          if (tid + x * kThreads < n && (!cut_k || place[x] < st.k)) mine += static_cast<double>(sh.c.q[tid + x * kThreads]);
        mine = cta_sum<kWarps>(mine, sh.d);
        if (cut_k)
          sum = mine;
        else
          done = mine >= sum * fmaxf(st.p, 0.f) * 1.000001;  // (else the cut lies behind them)
      }
      if (done) {
        unsigned long long best = 0ull;
        int bi = 0x7fffffff;
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
          const int i = tid + x * kThreads;
          if (i >= n) continue;
          const float l = logit_of(static_cast<uint32_t>(key[x] >> 32));
          const bool first = place[x] == 0;
          if ((cut_k && place[x] >= st.k) ||
              (cut_p && !first && static_cast<double>(before[x]) >= static_cast<double>(st.p) * sum) ||
              (!first && ex2((l - M) * c) < st.mp))
            continue;
          const unsigned long long o = exact_score(l, g[x], M, st.temp);
          const int t = static_cast<int>(~static_cast<uint32_t>(key[x]));
          if (o > best || (o == best && t < bi)) {
            best = o;
            bi = t;
          }
        }
        answer(best, bi);
      }
    }
  }
  if (!done && tid == 0) a.todo[atomicAdd(a.todo_n, 1u)] = row;
}

// ------------------------------------------------------------------ wide kernel

PE_DEV uint32_t row_addr(const void* local, uint32_t rank) {
  uint32_t remote;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
  return remote;
}
PE_DEV void put32(const void* local, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(row_addr(local, rank)), "r"(v) : "memory");
}
PE_DEV void put64(const void* local, uint32_t rank, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(row_addr(local, rank)), "l"(v) : "memory");
}
PE_DEV uint4 get128(const void* local, uint32_t rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(row_addr(local, rank))
               : "memory");
  return v;
}
// (all threads of all CTAs of the row)
PE_DEV void row_sync() {
  __syncwarp();
  cluster_sync_all();
}

// The last kept token of a row: those whose argmax_key is no less are kept.
struct Cut {
  unsigned long long key;
  double mass;  // weight of the kept ones, 2^-31
};

// Shared memory of a CTA of the wide kernel.  What the others of the row write or read there is
// held twice and taken in turn: whoever writes a place again has met all of them at a barrier
// since the last one read it.
struct __align__(16) WideShared {
  uint4 bins[2][kBins];  // count, sums of two or three parts of the weights' bits
  float m[kCluster], lo[kCluster];               // of every CTA: largest and least finite logit
  uint32_t least[2][kCluster], most[2][kCluster];  // ... orders of the cut's bin of the level before
  unsigned long long best[kCluster];
  int best_i[kCluster];
  Cands c;               // the tokens of the cut's bin, of all CTAs
  int tie;
  // this CTA's own
  unsigned long long scan_n[kWideWarps], scan_m[kWideWarps], k[kWideWarps];
  float wm[kWideWarps], wl[kWideWarps];
  uint32_t u[kWideWarps], v[kWideWarps];
  int i[kWideWarps];
  int digit, n_list;
  unsigned long long count, mass, n_in;
  uint32_t own, start;
};

// Sum over the CTA before this thread (wide kernel), and of all.
PE_DEV int wide_before(int v, int* warps, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = incl;
  __syncthreads();
  int before = incl - v;
  all = 0;
  for (int w = 0; w < kWideWarps; ++w) {
    if (w < warp) before += warps[w];
    all += warps[w];
  }
  return before;
}

template <typename T>
__global__ void __launch_bounds__(kWideThreads, 1) sample_wide_kernel(const SampleArgs a) {
  constexpr int kVec = 16 / sizeof(T);
  extern __shared__ uint4 held[];
  __shared__ WideShared sh;
  pdl_trigger();
  // (every CTA of the cluster has to have begun before another one writes to it)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  const uint32_t rank = blockIdx.x % kCluster;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = static_cast<int>(__ldcg(a.todo_n)), step = gridDim.x / kCluster;
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  uint32_t turn = 0;
  for (int item = blockIdx.x / kCluster; item < rows; item += step) {
    const int row = __ldcg(a.todo + item);
    const Settings st = a.set[row];
    const Row<T> s(a, row);
    const int nv = s.vectors(), per = (nv + kCluster - 1) / kCluster;
    const int v0 = min(static_cast<int>(rank) * per, nv), v1 = min(v0 + per, nv);
    auto get = [&](int v) { return a.resident ? held[v - v0] : s.load(v); };
    // two parts of a weight's 31 bits do where a bin of a slice has at most 2^16 tokens
    const bool small = per * kVec <= 65536;
    __syncthreads();
    // ---------------- the slice, its largest and least logit
    float m = -INFINITY, lo = INFINITY;
    for (int v = v0 + tid; v < v1; v += kUnroll * kWideThreads) {
      uint4 u[kUnroll];
#pragma unroll
      for (int x = 0; x < kUnroll; ++x)
        if (v + x * kWideThreads < v1) u[x] = s.load(v + x * kWideThreads);
#pragma unroll
      for (int x = 0; x < kUnroll; ++x)
        if (v + x * kWideThreads < v1) {
          if (a.resident) held[v + x * kWideThreads - v0] = u[x];
          float f[kVec];
          unpack16<T>(u[x], f);
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            m = fmaxf(m, f[e]);
            if (f[e] > -INFINITY) lo = fminf(lo, f[e]);
          }
        }
    }
    m = warp_max(m);
    lo = -warp_max(-lo);
    if (lane == 0) {
      sh.wm[warp] = m;
      sh.wl[warp] = lo;
    }
    __syncthreads();
    if (warp == 0) {
      m = warp_max(lane < kWideWarps ? sh.wm[lane] : -INFINITY);
      lo = -warp_max(lane < kWideWarps ? -sh.wl[lane] : -INFINITY);
      if (lane < kCluster) {
        put32(&sh.m[rank], lane, __float_as_uint(m));
        put32(&sh.lo[rank], lane, __float_as_uint(lo));
      }
    }
    row_sync();
    float M = -INFINITY;
    lo = INFINITY;
    for (int i = 0; i < kCluster; ++i) {
      M = fmaxf(M, sh.m[i]);
      lo = fminf(lo, sh.lo[i]);
    }
    const float c = scale_of(st.temp), it = 1.f / st.temp;
    auto weight_bits = [&](float x) { return static_cast<uint32_t>(ex2((x - M) * c) * 0x1p31f); };

    // ---------------- the cut: k tokens, and a share of the weight z (negative: of the row's)
    auto find = [&](int k, double share, double z) {
      Cut cut;
      // Digits, small ones first in the order: of the distance from the largest logit in bins
      // (an eighth of a factor 2 of weight each, or the row's range in kBins, whichever is finer:
      // the last takes all that is farther) and finer ones inside the last level's; if the cut's
      // bin stays too full without all in it being equal, of the bits of the logits' order.
      const float span = M - lo;
      float scale = span > 0.f && span < INFINITY ? fminf(kBins / span, 1e30f) : 0.f;
      if (share < 1.) scale = fmaxf(scale, fminf(8.f * c, 1e30f));
      double most = INFINITY;
      for (int bits = 0; bits < 2; ++bits) {
        int b0 = 0, b1 = 0;
        uint32_t prefix = 0;
        unsigned long long count = 0, mass = 0, n_in = ~0ull;
        uint32_t own = 0, start = 0;
        // the digit of a logit at this level, -1: it is not in the bins found so far
        auto digit = [&](float x, int level) {
          if (bits) {
            const uint32_t o = argmax_order(x);
            if (level > 0 && o >> (32 - 8 * level) != prefix >> (32 - 8 * level)) return -1;
            return static_cast<int>(255u - (o >> (24 - 8 * level) & 255u));
          }
          float t = (M - x) * scale;
          int b = min(kBins - 1, static_cast<int>(t));
          if (level > 0) {
            if (b != b0) return -1;
            t = (t - static_cast<float>(b)) * kBins;
            b = min(kBins - 1, static_cast<int>(t));
          }
          if (level > 1) {
            if (b != b1) return -1;
            t = (t - static_cast<float>(b)) * kBins;
            b = min(kBins - 1, static_cast<int>(t));
          }
          return b;
        };
        for (int level = 0; level < (bits ? 5 : 4); ++level) {
          // Counts and weights per digit (of the level behind the last: only whether all are equal)
          const bool last = level == (bits ? 4 : 3);
          uint4* bins = sh.bins[turn & 1];
          uint32_t (*word)[4] = reinterpret_cast<uint32_t (*)[4]>(bins);
          __syncthreads();
          for (int i = tid; i < kBins; i += kWideThreads) bins[i] = make_uint4(0, 0, 0, 0);
          __syncthreads();
          uint32_t least = 0xffffffffu, greatest = 0;
          for (int v = v0 + tid; v < v1; v += kWideThreads) {
            float f[kVec];
            unpack16<T>(get(v), f);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
              if (f[e] == -INFINITY) continue;
              const int d = last ? (digit(f[e], level - 1) == (bits ? 255 - static_cast<int>(prefix & 255u) : sh.digit) ? 0 : -1)
                                 : digit(f[e], level);
              if (d < 0) continue;
              if (level > 0) {
                const uint32_t o = argmax_order(f[e]);
                least = min(least, o);
                greatest = max(greatest, o);
              }
              if (last) continue;
              const uint32_t q = weight_bits(f[e]);
              atomicAdd(&word[d][0], 1u);
              if (small) {
                atomicAdd(&word[d][1], q & 0xffffu);
                atomicAdd(&word[d][2], q >> 16);
              } else {
                atomicAdd(&word[d][1], q & 0x7ffu);
                atomicAdd(&word[d][2], q >> 11 & 0x3ffu);
                atomicAdd(&word[d][3], q >> 21);
              }
            }
          }
          if (level > 0) {
            least = __reduce_min_sync(0xffffffffu, least);
            greatest = __reduce_max_sync(0xffffffffu, greatest);
            if (lane == 0) {
              sh.u[warp] = least;
              sh.v[warp] = greatest;
            }
            __syncthreads();
            if (warp == 0) {
              least = __reduce_min_sync(0xffffffffu, lane < kWideWarps ? sh.u[lane] : 0xffffffffu);
              greatest = __reduce_max_sync(0xffffffffu, lane < kWideWarps ? sh.v[lane] : 0u);
              if (lane < kCluster) {
                put32(&sh.least[turn & 1][rank], lane, least);
                put32(&sh.most[turn & 1][rank], lane, greatest);
              }
            }
          }
          row_sync();
          if (level > 0) {
            least = 0xffffffffu;
            greatest = 0;
            for (int i = 0; i < kCluster; ++i) {
              least = min(least, sh.least[turn & 1][i]);
              greatest = max(greatest, sh.most[turn & 1][i]);
            }
            if (least == greatest) {
              // ---------------- all in the cut's bin are equal: the first of them by index
              ++turn;
              const uint32_t q = weight_bits(logit_of(least));
              double t = fmin(static_cast<double>(n_in), static_cast<double>(k) - static_cast<double>(count));
              if (most < INFINITY && q > 0) t = fmin(t, ceil((most - static_cast<double>(mass)) / q));
              t = fmax(t, 1.);
              cut.key = static_cast<unsigned long long>(least) << 32;
              cut.mass = static_cast<double>(mass) + t * q;
              if (t >= static_cast<double>(n_in)) return cut;
              const int want = static_cast<int>(t) - static_cast<int>(start);  // the want-th of this CTA's
              if (want >= 1 && want <= static_cast<int>(own)) {
                int seen = 0;
                for (int vb = v0; vb < v1; vb += kWideThreads) {
                  const int v = vb + tid;
                  float f[kVec];
                  int eq = 0, all;
                  if (v < v1) {
                    unpack16<T>(get(v), f);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) eq += argmax_order(f[e]) == least;
                  }
                  int place = seen + wide_before(eq, sh.i, all);
                  seen += all;
                  if (v < v1 && place < want && place + eq >= want) {
#pragma unroll
                    for (int e = 0; e < kVec; ++e)
                      if (argmax_order(f[e]) == least && ++place == want)
                        for (int i = 0; i < kCluster; ++i) put32(&sh.tie, i, static_cast<uint32_t>(s.token(v) + e));
                  }
                }
              }
              row_sync();
              cut.key |= ~static_cast<uint32_t>(sh.tie);
              return cut;
            }
          }
          ++turn;
          if (last) break;
          // the row's sums per digit, and before it; thread t has digit t
          unsigned long long n_d = 0, m_d = 0;
          uint32_t mine = 0, before_me = 0;
          if (tid < kBins) {
            for (uint32_t i = 0; i < kCluster; ++i) {
              const uint4 w = get128(&bins[tid], i);
              n_d += w.x;
              m_d += small ? w.y + (static_cast<unsigned long long>(w.z) << 16)
                           : w.y + (static_cast<unsigned long long>(w.z) << 11) + (static_cast<unsigned long long>(w.w) << 21);
              if (i < rank) before_me += w.x;
              if (i == rank) mine = w.x;
            }
          }
          unsigned long long ni = n_d, mi = m_d;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long y0 = __shfl_up_sync(0xffffffffu, ni, o), y1 = __shfl_up_sync(0xffffffffu, mi, o);
            if (lane >= o) {
              ni += y0;
              mi += y1;
            }
          }
          if (lane == 31) {
            sh.scan_n[warp] = ni;
            sh.scan_m[warp] = mi;
          }
          if (tid == 0) sh.digit = -1;
          __syncthreads();
          unsigned long long cb = count + ni - n_d, mb = mass + mi - m_d, m_all = 0;
          for (int w = 0; w < kBins / 32; ++w) {
            if (w < warp) {
              cb += sh.scan_n[w];
              mb += sh.scan_m[w];
            }
            m_all += sh.scan_m[w];
          }
          // (the first token is kept whatever top_p is: nothing is before it)
          if (level == 0) most = share >= 1. ? INFINITY : fmax(share * (z >= 0. ? z : static_cast<double>(m_all)), 0.5);
          if (tid < kBins && n_d > 0 && cb < static_cast<unsigned long long>(k) && static_cast<double>(mb) < most)
            atomicMax(&sh.digit, tid);
          __syncthreads();
          if (tid == sh.digit) {
            sh.count = cb;
            sh.mass = mb;
            sh.n_in = n_d;
            sh.own = mine;
            sh.start = before_me;
            sh.n_list = 0;
          }
          __syncthreads();
          const int b = sh.digit;
          count = sh.count;
          mass = sh.mass;
          n_in = sh.n_in;
          own = sh.own;
          start = sh.start;
          if (n_in <= kList) {
            // ---------------- few: all of them to every CTA, their pairs compared
            for (int v = v0 + tid; v < v1; v += kWideThreads) {
              float f[kVec];
              unpack16<T>(get(v), f);
#pragma unroll
              for (int e = 0; e < kVec; ++e) {
                if (f[e] == -INFINITY || digit(f[e], level) != b) continue;
                const uint32_t at = start + atomicAdd(&sh.n_list, 1);
                const unsigned long long key = argmax_key(f[e], static_cast<uint32_t>(s.token(v) + e));
                const unsigned long long q = weight_bits(f[e]);
                for (int i = 0; i < kCluster; ++i) {
                  put64(&sh.c.key[at], i, key);
                  put64(&sh.c.q[at], i, q);
                }
              }
            }
            row_sync();
            const int n = static_cast<int>(n_in);
            unsigned long long key = 0, before = 0;
            int place = 0;
            if (tid < n) key = sh.c.key[tid];
            if ((tid & ~31) < n) {
              for (int j = 0; j < n; ++j)
                if (sh.c.key[j] > key) {
                  ++place;
                  before += sh.c.q[j];
                }
            }
            // the last that is kept
            const bool keep = tid < n && count + place < static_cast<unsigned long long>(k) &&
                              (place == 0 || static_cast<double>(mass + before) < most);
            const int kept = __syncthreads_count(keep);
            if (keep && place == kept - 1) {
              sh.count = key;
              sh.mass = mass + before + sh.c.q[tid];
            }
            __syncthreads();
            cut.key = sh.count;
            cut.mass = static_cast<double>(sh.mass);
            __syncthreads();
            return cut;
          }
          if (bits)
            prefix |= static_cast<uint32_t>(255 - b) << (24 - 8 * level);
          else if (level == 0)
            b0 = b;
          else if (level == 1)
            b1 = b;
        }
      }
      return cut;  // (not reached: tokens with the same four digits are equal)
    };

    const bool cut_k = st.k > 0, cut_p = st.p < 1.f;
    Cut cut{0ull, -1.};
    if (cut_k) cut = find(st.k, 1., -1.);
    if (cut_p) cut = find(cut_k ? st.k : 0x7fffffff, static_cast<double>(st.p), cut.mass);

    // ---------------- race over the slice's kept tokens
    const Noise<T> noise(a, row, s.shift);
    float bs = -INFINITY, bx = 0.f, bg = 0.f;
    int bi = 0x7fffffff;
    for (int v = v0 + tid; v < v1; v += kWideThreads) {
      float f[kVec], g[kVec];
      unpack16<T>(get(v), f);
      const int t0 = s.token(v);
      bool any = false;
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        if (argmax_key(f[e], static_cast<uint32_t>(t0 + e)) < cut.key ||
            (st.mp > 0.f && f[e] != M && ex2((f[e] - M) * c) < st.mp))
          f[e] = -INFINITY;
        any |= f[e] > -INFINITY;
      }
      if (!any) continue;
      noise.load(t0, a.V, g);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const float sc = f[e] > -INFINITY ? fmaf(f[e] - M, it, g[e]) : -INFINITY;
        if (sc > bs) {
          bs = sc;
          bi = t0 + e;
          bx = f[e];
          bg = g[e];
        }
      }
    }
    // (as in the row kernel: within reach, in 64 bits)
    const float wt = warp_max(bs);
    __syncthreads();
    if (lane == 0) sh.wm[warp] = wt;
    __syncthreads();
    float top = sh.wm[0];
    for (int w = 1; w < kWideWarps; ++w) top = fmaxf(top, sh.wm[w]);
    unsigned long long best = 0ull;
    if (bs > -INFINITY && (bs >= top || bs >= top - 1e-6f * (fabsf(top) + fabsf(bs) + 128.f)))
      best = exact_score(bx, bg, M, st.temp);
    else
      bi = 0x7fffffff;
    cta_best<kWideWarps>(best, bi, sh.k, sh.i);
    if (tid == 0) {
      put64(&sh.best[rank], 0, best);
      put32(&sh.best_i[rank], 0, static_cast<uint32_t>(bi));
    }
    row_sync();
    if (rank == 0 && warp == 0) {
      best = lane < kCluster ? sh.best[lane] : 0ull;
      bi = lane < kCluster ? sh.best_i[lane] : 0x7fffffff;
      warp_best(best, bi);
      if (lane == 0) {
        a.token[row] = best ? bi : -1;
        if (!best) set_status(a.status, PE_ST_SAMPLING);
      }
    }
  }
}

// ------------------------------------------------------------------ host

size_t al256(size_t x) { return (x + 255) / 256 * 256; }

constexpr int kSlice = 176 * 1024;   // of a row, in a CTA of the wide kernel
constexpr int kMaxParts = kGroups / (kThreads >> 5);

// Parts of a row: one wave of CTAs (four an SM) where the rows are few, at most 64 KB and at
// least a vector per thread each.
void plan(SampleArgs& a, int esize, int num_sms) {
  const int vec = 16 / esize;
  const int nvec = (a.V + 2 * (vec - 1)) / vec;  // whatever the row's place on the grid
  int parts = a.T <= 4 * num_sms ? 4 * num_sms / std::max(a.T, 1) : 1;
  parts = std::max(parts, (nvec * 16 + kMaxPartBytes - 1) / kMaxPartBytes);
  parts = std::min(parts, (nvec + kThreads - 1) / kThreads);
  parts = std::max(1, std::min(parts, kMaxParts));
  a.part = (nvec + parts - 1) / parts;
  a.parts = (nvec + a.part - 1) / a.part;
  a.gshift = 0;
  while (a.parts * (kThreads >> a.gshift) > kGroups) ++a.gshift;
}

// the most parts and groups of a row for any number of rows
size_t max_parts(int V) {
  return std::min<size_t>((static_cast<size_t>(V) + 6) / (4 * kThreads) + 1, kMaxParts);
}

template <typename T>
cudaError_t launch(const SampleArgs& a, int num_sms, cudaStream_t st) {
  // the function's shared-memory limit, once per device (a bit each; past 63 every time)
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (!(set.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(sample_wide_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSlice);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_release);
  }
  e = launch_chained(sample_row_kernel<T>, dim3(static_cast<unsigned>(a.T) * a.parts), dim3(kThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  e = launch_chained(sample_cut_kernel<T>, dim3(a.T), dim3(kThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  const int64_t slice = ((a.V + 7ll) * sizeof(T) / 16 + kCluster) / kCluster * 16 + 16;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster * std::min(a.T, std::max(num_sms / kCluster, 1)));
  cfg.blockDim = dim3(kWideThreads);
  cfg.dynamicSmemBytes = a.resident ? static_cast<size_t>(slice) : 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[3];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
  attr[1].val.sharedMemCarveout = cudaSharedmemCarveoutMaxShared;
  attr[2].id = cudaLaunchAttributeClusterDimension;
  attr[2].val.clusterDim.x = kCluster;
  attr[2].val.clusterDim.y = 1;
  attr[2].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 3;
  return cudaLaunchKernelEx(&cfg, sample_wide_kernel<T>, a);
}

}  // namespace
}  // namespace pe

using namespace pe;

extern "C" size_t pe_sample_workspace_bytes(int max_batch, int max_rows, int vocab) {
  if (max_batch < 0 || max_rows < 0 || vocab < 1 || vocab > 1 << 24) return 0;
  const size_t T = max_rows, parts = max_parts(vocab);
  return 256 + al256(T * sizeof(Settings)) + al256(T * sizeof(int32_t)) + al256(T * parts * sizeof(Part)) +
         al256(T * std::min<size_t>(parts * kThreads, kGroups) * sizeof(float));
}

extern "C" int pe_sample(int B, int T, const int32_t* qsl, const void* logits, int64_t ld_logits, int vocab, int dtype,
                         const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                         const float* gumbel, int64_t ld_gumbel, int32_t* token, void* ws, size_t ws_bytes,
                         void* stream) {
  NvtxRange nvtx("pe_sample");
  if (B < 0 || T < 0 || vocab < 1 || ld_logits < vocab || ld_gumbel < vocab) return PE_ERR_ARG;
  if (dtype != PE_DTYPE_F32 && dtype != PE_DTYPE_BF16) return PE_ERR_UNSUPPORTED;
  if (B == 0) return T == 0 ? PE_OK : PE_ERR_ARG;
  if (B > 65535 || vocab > 1 << 24) return PE_ERR_UNSUPPORTED;
  if (!qsl || !ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0 ||
      ws_bytes < pe_sample_workspace_bytes(B, T, vocab))
    return PE_ERR_ARG;
  const int esize = dtype == PE_DTYPE_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % esize != 0) return PE_ERR_ARG;
  for (const void* p : {static_cast<const void*>(qsl), static_cast<const void*>(temperature),
                        static_cast<const void*>(top_k), static_cast<const void*>(top_p),
                        static_cast<const void*>(min_p), static_cast<const void*>(gumbel),
                        static_cast<const void*>(token)})
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return PE_ERR_ARG;
  if (T == 0) return PE_OK;
  if (!logits || !gumbel || !token) return PE_ERR_ARG;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return PE_ERR_CUDA;
  SampleArgs a = {};
  a.B = B;
  a.T = T;
  a.V = vocab;
  a.qsl = qsl;
  a.logits = logits;
  a.ld = ld_logits;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.gumbel = gumbel;
  a.ld_g = ld_gumbel;
  a.token = token;
  plan(a, esize, sms);
  if (static_cast<int64_t>(T) * a.parts > 0x7fffffff) return PE_ERR_UNSUPPORTED;
  a.resident = (static_cast<int64_t>(vocab) + 7) * esize / 16 + kCluster <= static_cast<int64_t>(kSlice) / 16 * kCluster - kCluster;
  char* w = static_cast<char*>(ws);
  a.status = reinterpret_cast<uint32_t*>(w);
  a.todo_n = reinterpret_cast<uint32_t*>(w + 128);
  w += 256;
  a.set = reinterpret_cast<Settings*>(w);
  w += al256(T * sizeof(Settings));
  a.todo = reinterpret_cast<int32_t*>(w);
  w += al256(T * sizeof(int32_t));
  a.stat = reinterpret_cast<Part*>(w);
  w += al256(static_cast<size_t>(T) * a.parts * sizeof(Part));
  a.top = reinterpret_cast<float*>(w);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == PE_DTYPE_F32 ? launch<float>(a, sms, st) : launch<bf16>(a, sms, st);
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}
