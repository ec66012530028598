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
//                leaves the largest logit of each group of some dozens of tokens: what a few
//                neighbouring threads load in one trip, so that a group lies in few pieces.
//   cut kernel   a CTA per row joins the parts.  For a row with a cut:
//                  - a bound from below for it.  The groups' largest logits are tokens of the
//                    row, so the value at which k of them (for top-p: enough of them to weigh
//                    p of the whole) are reached cannot lie above the cut;
//                  - the tokens from the bound on, read again from the few groups that have
//                    one, in order; sums of their weights, the cut, the best score.
//   wide kernel  takes the rows for which that does not do (flat rows that keep thousands of
//                tokens, a large k, many equal logits), a cluster of CTAs a row with a slice
//                each in shared memory, beside its noise where that fits.  Top-p: all tokens race, and the
//                weight before the winner tells whether it is kept (if not, the tokens before it
//                race again).
//                Top-k: a histogram of counts over the distance from the largest logit, finer
//                ones inside the bin of the cut, then the race.  Weights are 40-bit integers there:
//                their sums do not depend on an order.
//
// The first kernel is bound by the logits' bytes, the others by the latency of a row's steps.
// Launched cold, 512 bf16 rows of 201,088 of mixed settings (245 MB with the noise): 46 us at 5.4
// TB/s, 18, and 25 for a dozen flat rows; 94 us a call.  8 fp32 rows: 7, 11 and 4, 12.5 us a
// call.  512 flat bf16 rows: 297 us, some 9 a row and cluster.  A flat row alone takes 15: a third is
// the first fetch of the code.
// Every row by a cluster with the row in shared memory took 162 us for 512 bf16 rows with top-k:
// the barriers of a row are waited for with its 400 KB held.  The cut in the first kernel, by a
// cluster of a row's CTAs, took 78 where the two took 72, the cut by the first CTA of the wide
// kernel's cluster for few rows 14.6 where three kernels took 13.4, by the last CTA of a row to
// finish 16.8 for 13.6.  Scores are compared in fp32,
// and in 64 bits only where two are near: a comparison in doubles takes 5000 clocks.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "pe_paged.h"
#include "pe_sampling.cuh"

namespace pe {
namespace {

constexpr int kThreads = 256;         // row kernel (the cut kernel counts on 2^8)
constexpr int kWarps = kThreads / 32;
constexpr int kChecked = kThreads - 32;  // requests whose offsets a CTA of the row kernel checks at a time
constexpr int kUnroll = 4;            // 16-byte loads in flight per thread
// of a row, per CTA (768 greedy bf16 rows of 201,088 74 us, 82 with 64 KB, 79 with 112; 384 fp32
// ones of 151,936 60, 62 and 61)
constexpr int kMaxPartBytes = 80 * 1024;
constexpr int kGroups = 4096;         // of a row, at most

constexpr int kCutBins = 512;         // cut kernel: of the groups' largest logits
constexpr int kList = 512;            // candidates of a row that are put in order
constexpr int kGroupList = 1024;      // groups that are read again, and vectors of theirs that matter

constexpr int kWideThreads = 512;     // wide kernel
constexpr int kWideWarps = kWideThreads / 32;
constexpr int kCluster = 8;
constexpr int kBins = 1024;           // two per thread
// The cut of a top-p row is looked for once kTries + 1 races are lost.  Each lost one leaves the weight before its
// winner, half of the rest on average, so top_p = 0.1 is reached in some three (512 flat bf16 rows of 201,088:
// 2390 us with kTries = 1, 1491 with 4, 1367 with 6, 1327 with 12; top_p = 0.5 1170, 799, 787, 786; 0.9 606 with
// any).  Near top_p = 0.01 alone fewer are faster (1527 us with 0, 1946 with 6).
constexpr int kTries = 6;

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
  int trips;         // of a part's CTA
  int gshift;        // threads of a group: 1 << gshift
  Part* stat;        // [T][parts]
  float* top;        // [T][parts][trips][kThreads >> gshift]
  Settings* set;  // [T] of each row
  uint32_t* todo_n;  // rows for the wide kernel
  int32_t* todo;     // [T]
  int resident;      // the wide kernel's slices fit in shared memory
  int near;          // ... beside their noise
  int checks, checked;  // CTAs of the row kernel that look at the requests' offsets, requests of each
};

struct Settings {
  float temp, p, mp;  // temperature (negative: a row of no request); top-p, 1: off; min-p, 0: off, at most 1
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
  if (s.mp > 1.f) {            // no weight reaches it: the first token, which is always kept
    s.k = a.V > 1;
    s.p = 1.f;
    s.mp = 0.f;
  }
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

// Half of a 32-byte sector whose other half is loaded next: by way of the L1 cache, past which every
// sector would come twice (512 bf16 rows of 201,088 without a cut 179 us, 145 like this).
PE_DEV uint4 ld_half16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
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
      for (int e = 0; e < kVec; e += 4) unpack16<float>(kVec > 4 ? ld_half16(g + t0 + e) : ld_stream16(g + t0 + e), x + e);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) x[e] = t0 + e >= 0 && t0 + e < V ? g[t0 + e] : 0.f;
    }
  }
};

// element e of a vector, as the bits of a float
template <typename T>
PE_DEV uint32_t element(const uint4& u, int e) {
  if (sizeof(T) == 4) return e == 0 ? u.x : e == 1 ? u.y : e == 2 ? u.z : u.w;
  const uint32_t w = e < 2 ? u.x : e < 4 ? u.y : e < 6 ? u.z : u.w;
  return e & 1 ? w & 0xffff0000u : w << 16;
}

PE_DEV unsigned long long exact_score(float x, float g, float M, float temp) {
  return score_order((static_cast<double>(x) - static_cast<double>(M)) / static_cast<double>(temp) + g);
}

// Whether a score may be the best one that rounds to `top` in fp32 (a score's rounding is 2^-23
// of its terms; noise past 128 is infinite).
PE_DEV bool within_reach(float score, float top, float term = 0.f) {
  return score > -INFINITY && (score >= top || score >= top - 1e-6f * (fabsf(top) + fabsf(score) + fabsf(term) + 128.f));
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
  v = warps[threadIdx.x % W];
#pragma unroll
  for (int o = W / 2; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
// Sum over the CTA, in a fixed order; all threads get it.
template <int W, typename X>
PE_DEV X cta_sum(X v, X* warps) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
  __syncthreads();
  X s = 0;
  for (int w = 0; w < W; ++w) s += warps[w];
  return s;
}

// The least whole number that is not below share * sum, share in [0, 1): what is below the one
// is below the other.  (Doubles are slow here, two a clock and SM.)
PE_DEV unsigned long long share_of(float share, unsigned long long sum) {
  const unsigned long long p = static_cast<unsigned long long>(fmaxf(share, 0.f) * 0x1p64f);
  return __umul64hi(p, sum) + (p * sum != 0ull);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) sample_row_kernel(const SampleArgs a) {
  constexpr int kVec = 16 / sizeof(T);
  __shared__ float warp_m[kWarps];
  __shared__ unsigned long long warp_k[kWarps];
  __shared__ int warp_i[kWarps];
  __shared__ Settings set_sh;
  __shared__ uint32_t status_sh;
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
      if (r >= 0) x = settings_of(a, r, status);
      set_sh = x;
      status_sh = status;
    }
  } else if (blockIdx.x < a.checks) {  // the offsets of every request, of those that no row is looked up in too
    bool bad = false;
    const int r0 = static_cast<int>(blockIdx.x) * a.checked, r1 = min(r0 + a.checked, a.B);
    for (int r = r0 + tid - 32; r < r1; r += kChecked) bad |= request_rows(a.qsl, r, a.T).bad;
    if (bad) set_status(a.status, PE_ST_ROWS_RANGE);
  }
  __syncthreads();
  const Settings st = set_sh;
  if (part == 0 && tid == 0) {
    a.set[row] = st;
    if (status_sh) set_status(a.status, status_sh);
    if (row == 0) *a.todo_n = 0u;
  }
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
    // (16 tokens a thread and trip, as many as the registers hold: 512 fp32 rows of 201,088 164 us, 169
    // with 8)
    constexpr int kRaceUnroll = 16 / kVec;
    float g[kRaceUnroll][kVec];
    auto load_noise = [&](int j) {
#pragma unroll
      for (int x = 0; x < kRaceUnroll; ++x)
        if (j + x * kThreads < n) noise.load(s.token(v0 + j + x * kThreads), a.V, g[x]);
    };
    load_noise(tid);
    for (int j = tid; j < n; j += kRaceUnroll * kThreads) {
      float mn = m;
#pragma unroll
      for (int x = 0; x < kRaceUnroll; ++x) mn = max_nan(mn, vec_max<T>(u[x]));
      const float off = mn == -INFINITY ? 0.f : mn;
      if (mn > m && bs < INFINITY) bs = fmaf(m - mn, it, bs);
      m = mn;
#pragma unroll
      for (int x = 0; x < kRaceUnroll; ++x) {
        float f[kVec], best = -INFINITY;
        unpack16<T>(u[x], f);
#pragma unroll
        for (int e = 0; e < kVec; ++e) best = fmaxf(best, fmaf(f[e] - off, it, g[x][e]));
        if (j + x * kThreads < n && (best > bs || bv < 0)) {
          bs = fmaxf(bs, best);
          bv = j + x * kThreads;
        }
        // the next trip's are on their way (the first kUnroll vectors of logits were loaded above)
        constexpr bool kAbove = kUnroll > kRaceUnroll;
        static_assert(kUnroll == kRaceUnroll || kUnroll == 2 * kRaceUnroll, "");
        u[x] = kAbove && j == tid ? u[(x + kRaceUnroll) % kUnroll] : no_tokens<T>();
        const int jn = j + (x + kRaceUnroll) * kThreads;
        if (jn < n) {
          if (!kAbove || j != tid) u[x] = s.load(v0 + jn);
          noise.load(s.token(v0 + jn), a.V, g[x]);
        }
      }
    }
    out.m = cta_max<kWarps>(m, warp_m);
    // The threads whose best is within reach of the CTA's: if there is more than one token, they
    // compare in 64 bits (which is slow: the one that there mostly is does without).
    // (`far` finite, so that infinite noise stays)
    const float far = m == out.m ? 0.f : fmaxf((m - out.m) * it, -FLT_MAX);
    bs += far;
    float top = warp_max(bs);
    __syncthreads();
    if (lane == 0) warp_m[warp] = top;
    __syncthreads();
    top = warp_m[0];
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, warp_m[w]);
    unsigned long long k = 0ull;
    int bi = 0x7fffffff;
    float bx = 0.f, bg = 0.f;
    const bool in = bv >= 0 && fabsf(out.m) < INFINITY && within_reach(bs, top, far);
    const int n_in = __syncthreads_count(in);
    if (in) {
      float f[kVec], g[kVec];
      unpack16<T>(s.load(v0 + bv), f);
      const int t0 = s.token(v0 + bv);
      noise.load(t0, a.V, g);
      int left = 0;
#pragma unroll
      for (int e = 0; e < kVec; ++e) left += within_reach(fmaf(f[e] - m, it, g[e]) + far, top, far);
      const bool alone = n_in == 1 && left == 1;
      for (int e = 0; e < kVec; ++e) {
        if (!within_reach(fmaf(f[e] - m, it, g[e]) + far, top, far)) continue;
        const unsigned long long o = alone ? 1ull : exact_score(f[e], g[e], out.m, st.temp);
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
    if (n_in > 1) cta_best<kWarps>(best, winner, warp_k, warp_i);
    out.idx = best ? winner : -1;
    // (its thread writes the part)
    if (n_in == 1 ? in : best ? bi == winner : tid == 0) {
      out.x = bx;
      out.g = bg;
      a.stat[static_cast<size_t>(row) * a.parts + part] = out;
    }
  } else {
    // sum of 2^((l - m) c), c = log2(e) / T, for top-p alone: the difference is exact near the
    // largest logit
    const bool weigh = st.k == 0 && st.p < 1.f;
    const float c = scale_of(st.temp);
    const uint64_t c2 = pack_f32x2(c, c);
    float sum = 0.f;
    float* top = a.top + (static_cast<size_t>(row) * a.parts + part) * a.trips * (kThreads >> a.gshift);
    for (int trip = 0; trip < a.trips; ++trip) {
      float of_trip = -INFINITY;
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) of_trip = max_nan(of_trip, vec_max<T>(u[x]));
      const float mn = max_nan(m, of_trip), off = mn == -INFINITY ? 0.f : mn;
      if (weigh) sum *= ex2((m - off) * c);  // one rescaling for the kUnroll vectors
      m = mn;
      const uint64_t off2 = pack_f32x2(-off, -off);
      uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) {
        float f[kVec];
        unpack16<T>(u[x], f);
        const int jn = tid + ((trip + 1) * kUnroll + x) * kThreads;
        u[x] = jn < n ? s.load(v0 + jn) : no_tokens<T>();
        if (weigh) {
#pragma unroll
          for (int e = 0; e < kVec; e += 2) {
            float p, q;
            unpack_f32x2(mul_f32x2(add_f32x2(pack_f32x2(f[e], f[e + 1]), off2), c2), p, q);
            acc[e / 2 & 1] = add_f32x2(acc[e / 2 & 1], pack_f32x2(ex2(p), ex2(q)));
          }
        }
      }
      float s0, s1;
      unpack_f32x2(add_f32x2(acc[0], acc[1]), s0, s1);
      sum += s0 + s1;
      for (int o = 1; o < 1 << a.gshift; o <<= 1) of_trip = max_nan(of_trip, __shfl_xor_sync(0xffffffffu, of_trip, o));
      if ((lane & ((1 << a.gshift) - 1)) == 0) top[trip * (kThreads >> a.gshift) + (tid >> a.gshift)] = of_trip;
    }
    out.m = cta_max<kWarps>(m, warp_m);
    if (weigh) out.s = cta_sum<kWarps>(m > -INFINITY ? sum * ex2((m - out.m) * c) : 0.f, warp_m);
  }
  if ((!free || st.temp == 0.f) && tid == 0) a.stat[static_cast<size_t>(row) * a.parts + part] = out;
}

// ------------------------------------------------------------------ cut kernel

// weights as integers: 2^38, so that 2^20 of them have a sum (in two parts: 2^20, 2^18)
constexpr float kOne = 0x1p38f;

// Shared memory of the cut kernel.
struct __align__(16) CutShared {
  float m[16];
  unsigned long long k[16], scan[16];
  int i[16], scan_n[16];
  int n, n_groups, n_vec, last, most, near;
  uint32_t bound;
  unsigned long long sum;
  float top[kGroups];
  union {
    struct {
      uint32_t cnt[kCutBins], least[kCutBins];  // of the groups' largest logits; order of the least
      uint32_t low[kCutBins], high[kCutBins];   // sums of their weights' lower 18 bits, and of the rest
    } h;
    struct {  // the candidates, and in order
      unsigned long long key[kList], sorted[kList];  // argmax_key: larger comes first
    } l;
  };
  uint16_t group[kGroupList];
  int vec[kGroupList];
};

// A weight, or a few together (at most 8), in units of 2^-40, truncated.  (Out of its bits: conversions
// between floats and 64-bit integers are two a clock and SM.)
PE_DEV unsigned long long as_weight(float w) {
  const uint32_t u = __float_as_uint(w);
  const unsigned long long m = static_cast<unsigned long long>((u & 0x7fffffu) | 0x800000u) << 20;
  return m >> min(130u - (u >> 23), 63u);  // (below 2^-86: 0)
}

// Sums over the CTA up to and with this thread (cut kernel); no barrier after the last read.
template <int W, typename T>
PE_DEV T sum_upto(T v, T* warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) warps[warp] = v;
  __syncthreads();
  T before = 0;
  for (int w = 0; w < W; ++w)
    if (w < warp) before += warps[w];
  return v + before;
}

// (for the rounding of a sum that is compared with another)
PE_DEV unsigned long long with_margin(unsigned long long x) { return x + (x >> 20); }

// The answer of a row from its parts.  16 warps, or 8 (with two bins and two candidates a thread)
// where the rows are more than the SMs hold of the former at once: 512 bf16 rows of 201,088 with top-k
// 69 us, 77 with 16 warps; 8 rows 19 and 20.
template <typename T, int W>
__global__ void __launch_bounds__(32 * W, 32 / W) sample_cut_kernel(const SampleArgs a) {
  constexpr int kVec = 16 / sizeof(T), kN = 32 * W, kE = kList / kN;
  static_assert(kCutBins == kList && kE * kN == kList && W <= 16, "");
  __shared__ CutShared sh;
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const Settings st = a.set[row];
  const Part* stat = a.stat + static_cast<size_t>(row) * a.parts;
  // (what only some rows need is asked for with the settings; no more parts than threads)
  const int gpt = 8 - a.gshift, groups = a.parts * a.trips << gpt;  // log2 of a trip's groups; the row's
  const float* top = a.top + static_cast<size_t>(row) * groups;
  float part_m = -INFINITY, part_s = 0.f, top_m[kGroups / kN];
  if (tid < a.parts) {
    part_m = __ldcg(&stat[tid].m);
    part_s = __ldcg(&stat[tid].s);
  }
#pragma unroll
  for (int x = 0; x < kGroups / kN; ++x)
    top_m[x] = tid + x * kN < groups ? __ldcg(top + tid + x * kN) : -INFINITY;
  auto answer = [&](unsigned long long k, int i) {
    cta_best<W>(k, i, sh.k, sh.i);
    if (tid == 0) {
      a.token[row] = k ? i : -1;
      if (!k) set_status(a.status, PE_ST_SAMPLING);
    }
  };
  if (st.temp < 0.f) return;
  if (st.temp == 0.f) {
    unsigned long long k = 0ull;
    for (int i = tid; i < a.parts; i += kN) k = max(k, __ldcg(&stat[i].key));
    answer(k, static_cast<int>(~static_cast<uint32_t>(k)));
    return;
  }
  const bool cut_k = st.k > 0, cut_p = st.p < 1.f, cut = cut_k || cut_p || st.mp > 0.f;
  float lo = INFINITY;
  if (cut) {
#pragma unroll
    for (int x = 0; x < kGroups / kN; ++x) {
      if (tid + x * kN < groups) sh.top[tid + x * kN] = top_m[x];
      if (top_m[x] > -INFINITY) lo = fminf(lo, top_m[x]);
    }
#pragma unroll
    for (int x = 0; x < kE; ++x) {
      sh.h.cnt[tid + x * kN] = 0;
      sh.h.least[tid + x * kN] = 0xffffffffu;
      sh.h.low[tid + x * kN] = sh.h.high[tid + x * kN] = 0;
    }
    if (tid == 0) {
      sh.n = sh.n_groups = sh.n_vec = 0;
      sh.last = kCutBins;
      sh.most = -1;
      sh.bound = 0xffffffffu;
    }
  }
  const float M = cta_max<W>(part_m, sh.m);
  if (!(fabsf(M) < INFINITY)) {  // no distribution
    answer(0ull, -1);
    return;
  }
  // the best score among the threads': where one alone is within reach, that one
  auto finish = [&](const bool* there, const float* l, const float* g, const int* t) {
    float score[kE], top = -INFINITY;
    bool in[kE];
    int near = 0;
#pragma unroll
    for (int x = 0; x < kE; ++x) {
      score[x] = !there[x] ? -INFINITY : g[x] < INFINITY ? fmaf(l[x] - M, 1.f / st.temp, g[x]) : g[x];
      top = fmaxf(top, score[x]);
    }
    top = cta_max<W>(top, sh.m);
#pragma unroll
    for (int x = 0; x < kE; ++x) {
      in[x] = there[x] && within_reach(score[x], top);
      near += __syncthreads_count(in[x]);
    }
    unsigned long long k = 0ull;
    int i = 0x7fffffff;
#pragma unroll
    for (int x = 0; x < kE; ++x) {
      if (!in[x]) continue;
      const unsigned long long o = near == 1 ? 1ull : exact_score(l[x], g[x], M, st.temp);
      if (o > k || (o == k && t[x] < i)) {
        k = o;
        i = t[x];
      }
    }
    if (near != 1)
      answer(k, i);
    else if (k)
      a.token[row] = i;
  };
  bool keep[kE];
  float l[kE], g[kE];
  int t[kE];
  if (!cut) {
#pragma unroll
    for (int x = 0; x < kE; ++x) {
      t[x] = x == 0 && tid < a.parts ? __ldcg(&stat[tid].idx) : -1;
      keep[x] = t[x] >= 0;
      l[x] = keep[x] ? __ldcg(&stat[tid].x) : 0.f;
      g[x] = keep[x] ? __ldcg(&stat[tid].g) : 0.f;
    }
    finish(keep, l, g, t);
    return;
  }
  const float c = scale_of(st.temp);
  // ---------------- a bound from below for the cut
  float bound = -INFINITY;
  unsigned long long z = 0;  // the weight of the whole row, where top-p alone asks for it
  if (cut_k || cut_p) {
    if (!cut_k)
      z = cta_sum<W>(
          part_m > -INFINITY ? static_cast<unsigned long long>(part_s * ex2((part_m - M) * c) * kOne) : 0ull, sh.k);
    // bins of the range that the groups' largest logits span
    lo = -cta_max<W>(-lo, sh.m);
    const float span = M - lo;
    const float scale = span > 0.f && span < INFINITY ? fminf(kCutBins / span, 1e30f) : 0.f;
    for (int i = tid; i < groups; i += kN) {
      const float t = sh.top[i], w = ex2((t - M) * c) * 0x1p20f;
      const uint32_t high = static_cast<uint32_t>(w);
      // (top-p alone: those that weigh next to nothing are left out, as many fall into one bin)
      if (t > -INFINITY && (cut_k || high > 0)) {
        const int b = min(kCutBins - 1, static_cast<int>((M - t) * scale));
        atomicAdd(&sh.h.cnt[b], 1u);
        atomicMin(&sh.h.least[b], argmax_order(t));
        if (!cut_k) {
          atomicAdd(&sh.h.high[b], high);
          atomicAdd(&sh.h.low[b], static_cast<uint32_t>((w - static_cast<float>(high)) * 0x1p18f));
        }
      }
    }
    __syncthreads();
    // The first bin with which there are k, or p of the weight (a margin for the rounding of
    // the sum); for want of the latter as many as are put in order: their weight tells, below.
    // (bins kE tid and on)
    uint32_t least[kE];
    int cnt[kE], upto[kE], total = 0;
    bool enough[kE];
#pragma unroll
    for (int x = 0; x < kE; ++x) {
      least[x] = sh.h.least[kE * tid + x];
      cnt[x] = sh.h.cnt[kE * tid + x];
      total += cnt[x];
    }
    total = sum_upto<W, int>(total, sh.scan_n);
#pragma unroll
    for (int x = kE - 1; x >= 0; --x) {
      upto[x] = total;
      enough[x] = total >= st.k;
      total -= cnt[x];
    }
    if (!cut_k) {
      unsigned long long w[kE], mass = 0;
#pragma unroll
      for (int x = 0; x < kE; ++x) {
        w[x] = sh.h.low[kE * tid + x] + (static_cast<unsigned long long>(sh.h.high[kE * tid + x]) << 18);
        mass += w[x];
      }
      mass = sum_upto<W, unsigned long long>(mass, sh.scan);
      const unsigned long long need = with_margin(share_of(st.p, z));
      if (tid == kN - 1) sh.near = mass >= need - (need >> 2);
      int most = -1;
#pragma unroll
      for (int x = kE - 1; x >= 0; --x) {
        enough[x] = mass >= need;
        mass -= w[x];
        if (most < 0 && upto[x] <= kList / 2) most = kE * tid + x;
      }
      most = __reduce_max_sync(0xffffffffu, most);
      if (lane == 0) atomicMax(&sh.most, most);
    }
    int last = kCutBins;
#pragma unroll
    for (int x = kE - 1; x >= 0; --x)
      if (enough[x]) last = kE * tid + x;
    last = __reduce_min_sync(0xffffffffu, last);
    if (lane == 0) atomicMin(&sh.last, last);
    __syncthreads();
    const int bin = sh.last < kCutBins || cut_k ? sh.last : sh.most;
    uint32_t o = 0xffffffffu;
#pragma unroll
    for (int x = 0; x < kE; ++x)
      if (kE * tid + x <= bin) o = min(o, least[x]);
    o = __reduce_min_sync(0xffffffffu, o);
    if (lane == 0) atomicMin(&sh.bound, o);
    __syncthreads();
    // (where all groups' largest are far from enough, the tokens behind them weigh as much)
    if (bin < 0 || bin == kCutBins || sh.bound == 0xffffffffu || (sh.last == kCutBins && !sh.near)) {
      if (tid == 0) a.todo[atomicAdd(a.todo_n, 1u)] = row;
      return;
    }
    bound = logit_of(sh.bound);
  } else {
    // min-p alone: the logit that its weight stands for, a little less for the roundings
    bound = fminf(M + (log2f(st.mp) * 1.00001f - 1e-5f) / c, M);
  }
  // ---------------- the groups that have a token from the bound on, and those tokens
  for (int i = tid; i < groups; i += kN)
    if (sh.top[i] > -INFINITY && sh.top[i] >= bound) {
      const int at = atomicAdd(&sh.n_groups, 1);
      if (at < kGroupList) sh.group[at] = static_cast<uint16_t>(i);
    }
  __syncthreads();
  const Row<T> s(a, row);
  const int nv = s.vectors(), n_groups = sh.n_groups;
  if (n_groups <= kGroupList) {
    // Which of their vectors reach the bound (a group has those of its threads in each of a trip's
    // loads), a thread to a vector.  Then those vectors' tokens.
    const int per = 2 + a.gshift, items = n_groups << per;  // log2 of a group's vectors
    static_assert(kUnroll == 4 && kThreads == 256, "");
    for (int i0 = tid & ~31; i0 < items; i0 += kUnroll * kN) {
      uint4 u[kUnroll];
      int v[kUnroll];
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) {
        const int i = i0 + x * kN + lane;
        const int g = sh.group[min(i, items - 1) >> per], j = i & ((1 << per) - 1);
        const int trip = g >> gpt, part = trip / a.trips;
        const int at = (trip - part * a.trips) * kUnroll * kThreads + (j >> a.gshift) * kThreads +
                       ((g & ((1 << gpt) - 1)) << a.gshift) + (j & ((1 << a.gshift) - 1));
        v[x] = part * a.part + at;
        if (i >= items || at >= a.part || v[x] >= nv) v[x] = -1;
        u[x] = v[x] >= 0 ? s.load(v[x]) : no_tokens<T>();
      }
      unsigned hit[kUnroll];
      int hits = 0;
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) {
        hit[x] = __ballot_sync(0xffffffffu, v[x] >= 0 && vec_max<T>(u[x]) >= bound);
        hits += __popc(hit[x]);
      }
      int at = 0;
      if (lane == 0 && hits) at = atomicAdd(&sh.n_vec, hits);
      at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) {
        const int mine = at + __popc(hit[x] & ((1u << lane) - 1u));
        if ((hit[x] >> lane & 1u) && mine < kGroupList) sh.vec[mine] = v[x];
        at += __popc(hit[x]);
      }
    }
    __syncthreads();
    const int n_vec = sh.n_vec;
    for (int i0 = 0; i0 < min(n_vec, kGroupList); i0 += kN) {
      const int v = i0 + tid < min(n_vec, kGroupList) ? sh.vec[i0 + tid] : -1;
      const uint4 u = v >= 0 ? s.load(v) : no_tokens<T>();
      float f[kVec];
      unpack16<T>(u, f);
      unsigned some = 0;
#pragma unroll
      for (int e = 0; e < kVec; ++e) some |= (f[e] >= bound && f[e] > -INFINITY) << e;
      int upto = __popc(some);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      int at = 0;
      if (lane == 31 && upto) at = atomicAdd(&sh.n, upto);
      at = __shfl_sync(0xffffffffu, at, 31) + upto - __popc(some);
      for (; some; some &= some - 1, ++at) {
        const int e = __ffs(some) - 1, t = s.token(v) + e;
        if (at < kList) {
          sh.l.key[at] = argmax_key(__uint_as_float(element<T>(u, e)), static_cast<uint32_t>(t));
          // (its noise is asked for below)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(a.gumbel + row * a.ld_g + t));
        }
      }
    }
  }
  __syncthreads();
  const int n = sh.n;
  bool done = n_groups <= kGroupList && sh.n_vec <= kGroupList && n <= kList;
  if (done) {
    // ---------------- in order: each counts those before it; then thread i has the i-th
#pragma unroll 1
    for (int x = 0; x < kE; ++x) {
      const int i = tid + x * kN;
      const unsigned long long mine = i < n ? sh.l.key[i] : 0ull;
      int place = 0;
      if ((i & ~31) < n) {
#pragma unroll 8
        for (int j = 0; j < n; ++j) place += sh.l.key[j] > mine;
      }
      if (i < n) sh.l.sorted[place] = mine;
    }
    __syncthreads();
    float w[kE];
#pragma unroll
    for (int x = 0; x < kE; ++x) {
      const int i = kE * tid + x;
      const unsigned long long key = i < n ? sh.l.sorted[i] : 0ull;
      t[x] = static_cast<int>(~static_cast<uint32_t>(key));
      keep[x] = i < n && (!cut_k || i < st.k);
      g[x] = keep[x] ? a.gumbel[row * a.ld_g + t[x]] : 0.f;
      l[x] = logit_of(static_cast<uint32_t>(key >> 32));
      w[x] = ex2((l[x] - M) * c);
    }
    if (cut_p) {
      unsigned long long q[kE], mass = 0;
#pragma unroll
      for (int x = 0; x < kE; ++x) {
        q[x] = keep[x] ? as_weight(w[x]) >> 2 : 0ull;  // (kOne)
        mass += q[x];
      }
      mass = sum_upto<W, unsigned long long>(mass, sh.scan);
      if (tid == kN - 1) sh.sum = mass;
      __syncthreads();
      // (top-p alone: of all tokens, and if these do not weigh enough the cut lies behind them)
      const unsigned long long most = share_of(st.p, cut_k ? sh.sum : z);
      done = cut_k || sh.sum >= with_margin(most);
#pragma unroll
      for (int x = kE - 1; x >= 0; --x) {
        mass -= q[x];  // (before it)
        keep[x] = keep[x] && (kE * tid + x == 0 || mass < most);
      }
    }
    if (done) {
#pragma unroll
      for (int x = 0; x < kE; ++x) keep[x] = keep[x] && (kE * tid + x == 0 || w[x] >= st.mp);
      finish(keep, l, g, t);
      return;
    }
  }
  if (tid == 0) a.todo[atomicAdd(a.todo_n, 1u)] = row;
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
PE_DEV void put128(const void* local, uint32_t rank, uint4 v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(row_addr(local, rank)), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
// (all threads of all CTAs of the row)
PE_DEV void row_sync() {
  __syncwarp();
  cluster_sync_all();
}

// Shared memory of a CTA of the wide kernel.  What the others of the row write or read there is
// held twice and taken in turn: whoever writes a place again has met all of them at a barrier
// since the last one read it.
struct __align__(16) WideShared {
  uint2 bins[2][kBins];  // counts; or sums of weights, their lower and upper word
  float lo[kCluster];  // of every CTA: least finite logit
  uint4 in[2][kCluster];  // ... of the cut's bin: tokens, least and greatest order
  unsigned long long best[2][kCluster], best_key[2][kCluster];  // ... of its best score, and which token
  unsigned long long key[kList];  // the tokens of the cut's bin, of all CTAs
  int tie;
  // this CTA's own
  uint64_t full;  // (barrier) the slice is there
  int never;      // 0
  unsigned long long scan[kWideWarps], k[kWideWarps], mine[kList];
  float wm[kWideWarps];
  uint32_t u[kWideWarps], v[kWideWarps];
  int i[kWideWarps];
  int digit;
  uint32_t n_list;
  unsigned long long before;
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
// (two CTAs an SM, with half the registers: 512 mixed bf16 rows 159 us, 161 with one, 64 of them 91
// and 72)
__global__ void __launch_bounds__(kWideThreads, 1) sample_wide_kernel(const SampleArgs a) {
  constexpr int kVec = 16 / sizeof(T), kWideRace = 16 / kVec;  // (16 tokens a thread and trip)
  extern __shared__ uint4 held[];
  __shared__ WideShared sh;
  if (threadIdx.x == 0) {
    mbar_init(&sh.full, 1);
    sh.never = 0;
    fence_barrier_init();
  }
  pdl_trigger();
  // (every CTA of the cluster has to have begun before another one writes to it)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  const uint32_t rank = blockIdx.x % kCluster;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = static_cast<int>(__ldcg(a.todo_n)), step = gridDim.x / kCluster;
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  uint32_t turn = 0, fulls = 0;
  for (int item = blockIdx.x / kCluster; item < rows; item += step) {
    const int row = __ldcg(a.todo + item);
    const Settings st = a.set[row];
    const Row<T> s(a, row);
    const Noise<T> noise(a, row, s.shift);
    const bool cut_k = st.k > 0, cut_p = st.p < 1.f;
    const int nv = s.vectors(), per = (nv + kCluster - 1) / kCluster;
    const int v0 = min(static_cast<int>(rank) * per, nv), v1 = min(v0 + per, nv);
    // The slice, and the noise of all of it if there is no k: then all tokens race.  By bulk copies
    // what lies in whole vectors (all but the row's ends), of which this CTA has those up to w1.
    const bool near = a.near && noise.wide && !cut_k;
    uint4* held_g = held + per;
    auto inside = [&](int t0) { return t0 >= 0 && t0 + kVec <= a.V; };
    // (no more parts than threads)
    const float part_m = tid < a.parts ? __ldcg(&a.stat[static_cast<size_t>(row) * a.parts + tid].m) : -INFINITY;
    __syncthreads();
    if (a.resident) {
      const int w0 = v0 + (v0 < v1 && !inside(s.token(v0))), w1 = max(w0, v1 - (v0 < v1 && !inside(s.token(v1 - 1))));
      if (tid == 0) {
        const uint32_t bytes = static_cast<uint32_t>(w1 - w0) * 16u;
        fence_proxy_async();  // (the last row's slice has been read)
        mbar_arrive_expect_tx(&sh.full, near ? bytes * (1u + kVec / 4) : bytes);
        if (bytes) {
          bulk_load(held + w0 - v0, s.row + s.token(w0), bytes, &sh.full);
          if (near)
            bulk_load(held_g + (w0 - v0) * (kVec / 4), noise.g + s.token(w0), bytes * (kVec / 4), &sh.full);
        }
      } else if (tid < 3) {
        const int v = tid == 1 ? v0 : v1 - 1;
        if (v0 < v1 && (v < w0 || v >= w1)) held[v - v0] = s.load(v);
      }
    }
    auto get = [&](int v) { return a.resident ? held[v - v0] : s.load(v); };
    const float M = cta_max<kWideWarps>(part_m, sh.wm);
    if (a.resident) {
      if (!mbar_wait(&sh.full, fulls & 1, &sh.never)) {
        set_status(a.status, PE_ST_TIMEOUT);
        mbar_wait(&sh.full, fulls & 1, &sh.never);  // (no copy is in flight when the CTA leaves)
      }
      ++fulls;
    }
    // the row's least finite logit, for the bins of a k
    float lo = -INFINITY;
    if (cut_k) {
      lo = INFINITY;
      for (int v = v0 + tid; v < v1; v += kWideThreads) {
        float f[kVec];
        unpack16<T>(get(v), f);
#pragma unroll
        for (int e = 0; e < kVec; ++e) lo = f[e] > -INFINITY ? fminf(lo, f[e]) : lo;
      }
      lo = -cta_max<kWideWarps>(-lo, sh.wm);
      if (tid < kCluster) put32(&sh.lo[rank], tid, __float_as_uint(lo));
      row_sync();
      lo = -warp_max(-sh.lo[lane % kCluster]);
    }
    const float c = scale_of(st.temp), it = 1.f / st.temp;
    // 2^20 weights of at most 2^40 have a sum; what is cut off of them is below 2^-20 of it
    auto weight_of = [&](float x) { return as_weight(ex2((x - M) * c)); };
    auto add_weight = [](uint2& bin, unsigned long long q) {  // (the lower word's carry goes to the upper one)
      const uint32_t lo = static_cast<uint32_t>(q);
      const uint32_t hi = static_cast<uint32_t>(q >> 32) + (lo && atomicAdd(&bin.x, lo) + lo < lo);
      if (hi) atomicAdd(&bin.y, hi);
    };

    // A place in the order (an argmax_key, 0: the end), and whether a token comes no later.
    struct To {
      float x;
      int t;
    };
    auto place_of = [](unsigned long long key) {
      return To{key ? logit_of(static_cast<uint32_t>(key >> 32)) : -INFINITY,
                static_cast<int>(~static_cast<uint32_t>(key) & 0x7fffffffu)};
    };
    auto no_later = [](float l, int t, const To& to) { return (l > to.x) | ((l == to.x) & (t <= to.t)); };
    // The key of the best score among the tokens from a cut on, 0 if there is none.
    auto race = [&](unsigned long long cut) {
      const To to = place_of(cut);
      const bool all = cut == 0ull && !(st.mp > 0.f);
      // a vector's kept logits, -inf for the others; whether there are some
      auto light = [&](float l) { return l != M && ex2((l - M) * c) < st.mp; };
      auto kept = [&](int v, float* f) {
        const int t0 = s.token(v);
        unpack16<T>(v < v1 ? get(v) : no_tokens<T>(), f);
        if (all) return true;
        // (ties with the place apart, which are few: instructions are what a pass takes)
        bool any = false, tie = false;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          tie |= f[e] == to.x;
          f[e] = f[e] >= to.x ? f[e] : -INFINITY;
          any |= f[e] > -INFINITY;
        }
        if (tie) {
#pragma unroll
          for (int e = 0; e < kVec; ++e)
            if (f[e] == to.x && t0 + e > to.t) f[e] = -INFINITY;
        }
        if (st.mp > 0.f) {
#pragma unroll
          for (int e = 0; e < kVec; ++e)
            if (light(f[e])) f[e] = -INFINITY;
        }
        return any;
      };
      float bs = -INFINITY;
      int bv = -1;  // the vector with this thread's
      auto pass = [&](auto vectors, auto&& load) {
        constexpr int kV = decltype(vectors)::value;
        for (int v = v0 + tid; v < v1; v += kV * kWideThreads) {
          float f[kV][kVec], g[kV][kVec];
          bool any[kV];
#pragma unroll
          for (int x = 0; x < kV; ++x) {
            any[x] = kept(v + x * kWideThreads, f[x]);
            if (any[x]) load(v + x * kWideThreads, g[x]);
          }
#pragma unroll
          for (int x = 0; x < kV; ++x) {
            if (!any[x]) continue;
            float top = -INFINITY;
#pragma unroll
            for (int e = 0; e < kVec; ++e) top = fmaxf(top, fmaf(f[x][e] - M, it, g[x][e]));
            if (top > bs) {
              bs = top;
              bv = v + x * kWideThreads;
            }
          }
        }
      };
      if (near) {
        pass(std::integral_constant<int, 1>(), [&](int v, float* g) {
          if (inside(s.token(v))) {
#pragma unroll
            for (int e = 0; e < kVec / 4; ++e) unpack16<float>(held_g[(v - v0) * (kVec / 4) + e], g + 4 * e);
          } else {
            noise.load(s.token(v), a.V, g);
          }
        });
      } else {
        pass(std::integral_constant<int, kWideRace>(), [&](int v, float* g) { noise.load(s.token(v), a.V, g); });
      }
      const float wt = warp_max(bs);
      __syncthreads();
      if (lane == 0) sh.wm[warp] = wt;
      __syncthreads();
      float top = warp_max(sh.wm[lane % kWideWarps]);
      // The tokens within reach of the best score (of this thread's best vector).  As a rule it is
      // one in the whole row: then its fp32 score and key do, else the scores are formed again, in
      // 64 bits (as in the row kernel).
      for (bool exact = false;; exact = true) {
        const bool in = bv >= 0 && within_reach(bs, top);
        const int n_in = __syncthreads_count(in);
        // (a lane for each token of the vector)
        unsigned long long best = 0ull, key = 0ull;
        int bi = 0x7fffffff;
        unsigned found = 0;
        for (unsigned of = __ballot_sync(0xffffffffu, in); of; of &= of - 1) {
          const int v = __shfl_sync(0xffffffffu, bv, __ffs(of) - 1), t0 = s.token(v), e = lane & (kVec - 1);
          const float l = __uint_as_float(element<T>(get(v), e));
          bool there = lane < kVec && l > -INFINITY && no_later(l, t0 + e, to) && !(st.mp > 0.f && light(l));
          float g = 0.f;
          if (there) g = near && inside(t0) ? reinterpret_cast<const float*>(held_g)[(v - v0) * kVec + e] : noise.g[t0 + e];
          there = there && within_reach(fmaf(l - M, it, g), top);
          found |= __ballot_sync(0xffffffffu, there);
          const unsigned long long o = !there ? 0ull : exact ? exact_score(l, g, M, st.temp) : 1ull;
          if (o > best) {
            best = o;
            bi = t0 + e;
            key = argmax_key(l, static_cast<uint32_t>(bi));
          }
        }
        // its thread, or the first where there is none (key 0: of several), tells the others
        unsigned long long k = best;
        int i = bi;
        if (exact) cta_best<kWideWarps>(k, i, sh.k, sh.i);
        const bool alone = n_in == 1 && __popc(found) == 1;  // (of the warp with it)
        const bool tells = __syncthreads_or(alone) ? alone && best : exact && k ? bi == i && best == k : tid == 0;
        if (const unsigned teller = __ballot_sync(0xffffffffu, tells)) {
          if (!exact) {
            k = __float_as_uint(top);
            if (!alone) key = 0ull;
          }
          k = __shfl_sync(0xffffffffu, k, __ffs(teller) - 1);
          key = __shfl_sync(0xffffffffu, key, __ffs(teller) - 1);
          if (lane < kCluster) {
            put64(&sh.best[turn & 1][rank], lane, k);
            put64(&sh.best_key[turn & 1][rank], lane, key);
          }
        }
        row_sync();
        // (lane i: CTA i % kCluster's)
        k = sh.best[turn & 1][lane % kCluster];
        key = sh.best_key[turn & 1][lane % kCluster];
        ++turn;
        if (exact) {  // (equal scores: the lowest index)
          i = static_cast<int>(~static_cast<uint32_t>(key) & 0x7fffffffu);
          const unsigned long long mine = k;
          const int at = i;
          warp_best(k, i);
          return k ? __shfl_sync(0xffffffffu, key, __ffs(__ballot_sync(0xffffffffu, mine == k && at == i)) - 1) : 0ull;
        }
        const float theirs = __uint_as_float(static_cast<uint32_t>(k));
        top = warp_max(theirs);
        const unsigned ctas = __ballot_sync(0xffffffffu, lane < kCluster && within_reach(theirs, top));
        if (ctas == 0) return 0ull;
        key = __shfl_sync(0xffffffffu, key, __ffs(ctas) - 1);
        if ((ctas & (ctas - 1)) == 0 && key) return key;
      }
    };
    // Sums of two over the row; all threads get them.
    auto wide_sums = [&](unsigned long long& x, unsigned long long& y) {
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, o);
        y += __shfl_xor_sync(0xffffffffu, y, o);
      }
      __syncthreads();
      if (lane == 0) {
        sh.scan[warp] = x;
        sh.k[warp] = y;
      }
      __syncthreads();
      if (warp == 0) {
        x = lane < kWideWarps ? sh.scan[lane] : 0ull;
        y = lane < kWideWarps ? sh.k[lane] : 0ull;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          x += __shfl_xor_sync(0xffffffffu, x, o);
          y += __shfl_xor_sync(0xffffffffu, y, o);
        }
        if (lane < kCluster) {
          put64(&sh.best[turn & 1][rank], lane, x);
          put64(&sh.best_key[turn & 1][rank], lane, y);
        }
      }
      row_sync();
      x = sh.best[turn & 1][lane % kCluster];
      y = sh.best_key[turn & 1][lane % kCluster];
#pragma unroll
      for (int o = kCluster / 2; o; o >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, o);
        y += __shfl_xor_sync(0xffffffffu, y, o);
      }
      ++turn;
    };

    // ---------------- The cut: the last token with less than `most` tokens, or weight, before it.
    // Returns its argmax_key.
    auto find = [&](unsigned long long most, bool by_w) {
      // Digits, small ones first in the order: of the distance from the largest logit in bins (a
      // 32nd of a factor 2 of weight each, or the row's range in kBins, whichever is finer: the
      // last takes all that is farther) and finer ones inside the cut's; if that stays too full
      // without all in it being equal, ten bits of the logits' order at a time.
      constexpr float kTop = kBins - 1;
      // (0 .. kTop to the nearest integer: an addition that leaves it in the low bits)
      auto linear = [](float t) { return __float_as_int(t + 8388608.f) & (kBins - 1); };
      const float span = M - lo;
      float scale = span > 0.f && span < INFINITY ? fminf(kBins / span, 1e30f) : 0.f;
      if (by_w) scale = fmaxf(scale, fminf(32.f * c, 1e30f));
      for (int bits = 0; bits < 2; ++bits) {
        int b0 = 0, b1 = 0, b2 = 0, b3 = 0;
        unsigned long long before = 0;  // tokens, or weight, before the cut's bin
        // the bin of a logit at this level, -1: it is not in the bins found so far
        auto digit = [&](float x, int level) {
          if (bits) {
            const uint32_t o = ~argmax_order(x);
            if ((level > 0 && static_cast<int>(o >> 22) != b0) || (level > 1 && static_cast<int>(o >> 12 & 1023u) != b1) ||
                (level > 2 && static_cast<int>(o >> 2 & 1023u) != b2) || (level > 3 && static_cast<int>(o & 3u) != b3))
              return -1;
            return static_cast<int>(level == 0 ? o >> 22 : level == 1 ? o >> 12 & 1023u : level == 2 ? o >> 2 & 1023u : o & 3u);
          }
          const float t0 = fminf((M - x) * scale, kTop);
          int b = linear(t0);
          if (level == 0) return b;
          if (b != b0) return -1;
          float t = (t0 - static_cast<float>(b) + 0.5f) * kTop;
          b = linear(t);
          if (level > 1) {
            if (b != b1) return -1;
            t = (t - static_cast<float>(b) + 0.5f) * kTop;
            b = linear(t);
          }
          if (level > 2 && b != b2) return -1;
          return b;
        };
        const int levels = bits ? 4 : 3;
        for (int level = 0; level <= levels; ++level) {
          // Of the cut's bin of the level before: how many tokens, whether they differ, and the
          // first of them in a list; and the bins of this level.
          uint2* bins = sh.bins[turn & 1];
          __syncthreads();
          for (int i = tid; i < kBins; i += kWideThreads) bins[i] = make_uint2(0, 0);
          if (tid == 0) {
            sh.n_list = 0;
            sh.digit = -1;
          }
          __syncthreads();
          uint32_t least = 0xffffffffu, greatest = 0;
          if (level == 0 && !bits) {
            // (every token, without a branch)
            for (int v = v0 + tid; v < v1; v += kWideThreads) {
              float f[kVec];
              unpack16<T>(get(v), f);
#pragma unroll
              for (int e = 0; e < kVec; ++e) {
                const int d = linear(fminf((M - f[e]) * scale, kTop));
                if (by_w) {
                  add_weight(bins[d], weight_of(f[e]));
                } else if (f[e] > -INFINITY) {
                  atomicAdd(&bins[d].x, 1u);
                }
              }
            }
          } else {
            for (int v = v0 + tid; v < v1; v += kWideThreads) {
              float f[kVec];
              unpack16<T>(get(v), f);
              // which may be in the bins found so far: few are
              unsigned some = 0;
#pragma unroll
              for (int e = 0; e < kVec; ++e)
                some |= (f[e] > -INFINITY && (bits || fabsf(fminf((M - f[e]) * scale, kTop) - static_cast<float>(b0)) <= 0.5f))
                        << e;
              if (!some) continue;
#pragma unroll 1
              for (int e = 0; e < kVec; ++e) {
                if (!(some >> e & 1u)) continue;
                const uint32_t x = element<T>(get(v), e);
                const float l = __uint_as_float(x);
                const int d = digit(l, level);
                if (d < 0) continue;
                if (level > 0) {
                  const uint32_t o = argmax_order(l);
                  least = min(least, o);
                  greatest = max(greatest, o);
                  const uint32_t at = atomicAdd(&sh.n_list, 1u);
                  if (at < kList) sh.mine[at] = argmax_key(l, static_cast<uint32_t>(s.token(v) + e));
                }
                if (level == levels) continue;
                if (by_w) {
                  add_weight(bins[d], weight_of(l));
                } else {
                  atomicAdd(&bins[d].x, 1u);
                }
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
              if (lane < kCluster) put128(&sh.in[turn & 1][rank], lane, make_uint4(sh.n_list, least, greatest, 0u));
            }
          }
          row_sync();
          if (level > 0) {
            uint32_t n_in = 0, start = 0;
            least = 0xffffffffu;
            greatest = 0;
            for (uint32_t i = 0; i < kCluster; ++i) {
              const uint4 x = sh.in[turn & 1][i];
              if (i < rank) start += x.x;
              n_in += x.x;
              least = min(least, x.y);
              greatest = max(greatest, x.z);
            }
            const uint32_t own = sh.in[turn & 1][rank].x;
            if (least == greatest) {
              // ---------------- all are equal: the first ones by index
              ++turn;
              const unsigned long long q = by_w ? weight_of(logit_of(least)) : 1ull;
              const unsigned long long t = q > 0 ? (most - before + q - 1) / q : n_in;  // (before < most)
              const unsigned long long key = static_cast<unsigned long long>(least) << 32;
              if (t >= n_in) return key;
              const int want = static_cast<int>(t) - static_cast<int>(start);  // of this CTA's
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
              return key | ~static_cast<uint32_t>(sh.tie);
            }
            if (n_in <= kList) {
              // ---------------- few: to every CTA, their pairs compared
              ++turn;
              for (uint32_t i = tid; i < own * kCluster; i += kWideThreads)
                put64(&sh.key[start + i / kCluster], i % kCluster, sh.mine[i / kCluster]);
              row_sync();
              const unsigned long long key = tid < n_in ? sh.key[tid] : 0ull;
              unsigned long long ahead = before;
              sh.mine[tid] = by_w ? weight_of(logit_of(static_cast<uint32_t>(key >> 32))) : 1ull;
              __syncthreads();
              if ((tid & ~31) < n_in) {
                for (uint32_t j = 0; j < n_in; ++j)
                  if (sh.key[j] > key) ahead += sh.mine[j];
              }
              // the last that is kept (the first one always is)
              const bool keep = tid < n_in && ahead < most;
              unsigned long long last = keep ? ~key : 0ull;
#pragma unroll
              for (int o = 16; o; o >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
              __syncthreads();
              if (lane == 0) sh.k[warp] = last;
              __syncthreads();
              for (int w = 0; w < kWideWarps; ++w) last = max(last, sh.k[w]);
              return ~last;
            }
          }
          if (level == levels) {
            ++turn;
            break;
          }
          // the row's sums per bin, and before it; thread t has bins 2 t and 2 t + 1
          unsigned long long x0 = 0, x1 = 0;
          uint4 w[kCluster];
#pragma unroll
          for (uint32_t i = 0; i < kCluster; ++i) w[i] = get128(&bins[2 * tid], i);
#pragma unroll
          for (uint32_t i = 0; i < kCluster; ++i) {
            x0 += w[i].x + (static_cast<unsigned long long>(w[i].y) << 32);
            x1 += w[i].z + (static_cast<unsigned long long>(w[i].w) << 32);
          }
          ++turn;
          unsigned long long upto = x0 + x1;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
          }
          if (lane == 31) sh.scan[warp] = upto;
          __syncthreads();
          unsigned long long first = before + upto - x0 - x1;
          for (int w = 0; w < warp; ++w) first += sh.scan[w];
          // the last bin that is not empty and has a kept token
          const int b = x1 > 0 && first + x0 < most ? 2 * tid + 1 : x0 > 0 && first < most ? 2 * tid : -1;
          if (b >= 0) atomicMax(&sh.digit, b);
          __syncthreads();
          if (b >= 0 && b == sh.digit) sh.before = b & 1 ? first + x0 : first;
          __syncthreads();
          before = sh.before;
          (level == 0 ? b0 : level == 1 ? b1 : level == 2 ? b2 : b3) = sh.digit;
        }
      }
      return 0ull;  // (not reached: tokens of the same order are equal)
    };

    // ---------------- The best score among the tokens from a cut on (all CTAs get its key, 0: there
    // is none); for top-p, is that token kept?  If it is not, none behind it is: the tokens before
    // it race again.  Few are rejected, by the noise of a Gumbel draw; after kTries the cut is
    // looked for.
    unsigned long long cut = cut_k ? find(st.k, false) : 0ull, won = 0ull, most = 0ull;
    for (int attempt = 0;; ++attempt) {
      won = race(cut);
      if (!cut_p || won == 0ull || attempt > kTries) break;
      // the weight before it, and (once) of all that top-p is a share of
      unsigned long long before = 0ull, all = 0ull;
      const To last = place_of(cut);
      To to = place_of(won);
      --to.t;
      for (int v = v0 + tid; v < v1; v += kWideThreads) {
        float f[kVec];
        unpack16<T>(get(v), f);
        // (a vector's in fp32; the ties at a place apart, which are few)
        float q[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) q[e] = ex2((f[e] - M) * c);
        auto upto = [&](const To& to) {
          float w = 0.f;
          bool tie = false;
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            if (f[e] > to.x) w += q[e];
            tie |= f[e] == to.x;
          }
          if (tie) {
            const int t0 = s.token(v);
#pragma unroll
            for (int e = 0; e < kVec; ++e)
              if (f[e] == to.x && t0 + e <= to.t) w += q[e];
          }
          return as_weight(w);
        };
        before += upto(to);
        if (attempt == 0) all += upto(last);
      }
      wide_sums(before, all);
      // (the first token is kept whatever top_p is: nothing is before it)
      if (attempt == 0) most = max(share_of(st.p, all), 1ull);
      if (before < most) break;
      // (find adds up other roundings of the weights, of all tokens: no place behind the cut so far)
      cut = won + 1ull;
      if (attempt == kTries) cut = max(cut, find(most, true));
    }
    if (rank == 0 && tid == 0) {
      a.token[row] = won ? static_cast<int>(~static_cast<uint32_t>(won)) : -1;
      if (!won) set_status(a.status, PE_ST_SAMPLING);
    }
  }
}

// ------------------------------------------------------------------ host

size_t al256(size_t x) { return (x + 255) / 256 * 256; }

constexpr int kSlice = 200 * 1024;   // of a row and of its noise, in a CTA of the wide kernel
constexpr int kMaxParts = kGroups / (kThreads >> 5);  // (and trips, in all of a row's parts)
static_assert(kMaxParts <= 512 && kMaxParts <= kWideThreads, "");
constexpr int kMaxVocab = 1 << 20;
constexpr int kWave = 4;  // CTAs of the row kernel per SM

// Parts of a row: one wave of CTAs (four an SM) where the rows are few, at most kMaxPartBytes and
// at least a vector per thread each.
void plan(SampleArgs& a, int esize, int num_sms) {
  const int vec = 16 / esize;
  const int nvec = (a.V + 2 * (vec - 1)) / vec;  // whatever the row's place on the grid
  int parts = a.T <= kWave * num_sms ? kWave * num_sms / std::max(a.T, 1) : 1;
  parts = std::max(parts, (nvec * 16 + kMaxPartBytes - 1) / kMaxPartBytes);
  parts = std::min(parts, (nvec + kThreads - 1) / kThreads);
  parts = std::max(1, std::min(parts, kMaxParts));
  // (no more than kMaxParts trips, which are 2^21 logits: parts of whole ones where that matters)
  const int trip = kUnroll * kThreads;
  a.part = (nvec + parts - 1) / parts;
  if (static_cast<int64_t>((nvec + a.part - 1) / a.part) * ((a.part + trip - 1) / trip) > kMaxParts)
    a.part = (a.part + trip - 1) / trip * trip;
  a.parts = (nvec + a.part - 1) / a.part;
  a.trips = (a.part + kUnroll * kThreads - 1) / (kUnroll * kThreads);
  a.gshift = 0;
  while (a.gshift < 5 && a.parts * a.trips * (kThreads >> a.gshift) > kGroups) ++a.gshift;
}

// the most vectors of a slice, whatever the row's place on the grid
int64_t slice_vectors(int V, int esize) { return ((V + 7ll) * esize / 16 + kCluster) / kCluster + 1; }

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
  const bool many = a.T > 2 * num_sms && a.parts <= 256;
  e = launch_chained(many ? sample_cut_kernel<T, 8> : sample_cut_kernel<T, 16>, dim3(a.T), dim3(many ? 256 : 512), 0, st,
                     a);
  if (e != cudaSuccess || !(a.top_k || a.top_p || a.min_p)) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster * std::min(a.T, std::max(num_sms / kCluster, 1)));
  cfg.blockDim = dim3(kWideThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(a.near ? slice_vectors(a.V, sizeof(T)) * (16 + 64 / sizeof(T))
                                             : a.resident ? slice_vectors(a.V, sizeof(T)) * 16 : 0);
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
  if (max_batch < 0 || max_rows < 0 || vocab < 1 || vocab > kMaxVocab) return 0;
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
  if (B > 65535 || vocab > kMaxVocab) return PE_ERR_UNSUPPORTED;
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
  a.checked = std::max(kChecked, (B - 1) / (T * a.parts) + 1);
  a.checks = (B + a.checked - 1) / a.checked;
  a.resident = slice_vectors(vocab, esize) * 16 <= kSlice;
  a.near = slice_vectors(vocab, esize) * (16 + 64 / esize) <= kSlice;
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
