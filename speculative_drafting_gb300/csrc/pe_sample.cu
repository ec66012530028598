// The target's token after each row: temperature, top-k, top-p, min-p, from given noise
// (pe_sample).
//
// The kept tokens are the first ones of one order (logit descending, index ascending), as many
// as all three settings allow, so a row's answer needs the place of the cut in that order and
// then the best of (l - max) / T + g over the tokens before it.  Nothing is sorted as a whole.
//
// One cluster of CTAs per row, each with a slice of the row in shared memory: the logits are
// read once.
//   1. Largest logit of the row; each thread's largest one of its share of the slice.
//   2. A bound from below for the cut: the threads' largest values are tokens of the row, so
//      the value at which k of them (for top-p: enough of them to weigh p of the whole) are
//      reached cannot lie above the cut.  They go into kBins bins, a bin of the range that they
//      span each.
//   3. The tokens from the bound on, some more than are kept, go to the first CTA with their
//      noise: rank and weight before each by comparing all pairs, the cut, the best score.
// Where that does not do (a flat row that keeps thousands, a large k, many equal logits),
// the cut is found digit by digit: histograms of counts and weights over 8 bits of the
// logits' order at a time, weights as 31-bit integers (their sums do not depend on the
// order), then all CTAs race over their slices.
//
// Rows without cuts (and greedy ones) need neither 2 nor 3.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "pe_paged.h"
#include "pe_sampling.cuh"

namespace pe {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 64;
constexpr int kList = 512;   // candidates of a row that the first CTA compares
constexpr int kUnroll = 4;   // 16-byte loads in flight per thread
constexpr int kDigits = 256;

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
  int ctas;      // of a row
  int resident;  // slices stay in shared memory
};

// What a CTA of the cluster tells the others, in their shared memory.
struct FromCta {
  float m, lo;     // largest logit; least finite of the threads' largest
  int cand;        // candidates
  double z;        // sum of weights
  uint32_t cnt[kBins], least[kBins];  // threads' largest values per bin; order of their least
  unsigned long long mass[kBins];     // their weights, 2^-40
};

struct Entry {
  unsigned long long key;  // order of the logit, then of the index: larger comes first
  float g;
};

struct Best {
  unsigned long long order;
  int idx;
};

union Scratch {
  FromCta from[kMaxCluster];
  // [two levels in turn][digit]: count, and the sums of three parts of the weights' bits
  uint32_t digits[2][kDigits][4];
};

PE_DEV uint32_t cluster_addr(const void* local, uint32_t rank) {
  uint32_t remote;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
  return remote;
}
PE_DEV void put32(const void* local, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(local, rank)), "r"(v) : "memory");
}
PE_DEV void put64(const void* local, uint32_t rank, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_addr(local, rank)), "l"(v) : "memory");
}
PE_DEV uint32_t get32(const void* local, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(local, rank)) : "memory");
  return v;
}
PE_DEV uint32_t add32(const void* local, uint32_t rank, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;"
               : "=r"(old)
               : "r"(cluster_addr(local, rank)), "r"(v)
               : "memory");
  return old;
}

// (all threads of all CTAs of the row)
PE_DEV void row_sync() {
  __syncwarp();
  cluster_sync_all();
}

// The logit of an order (argmax_order), and one that is in none of its values
PE_DEV float logit_of(uint32_t order) {
  return __uint_as_float(order & 0x80000000u ? order & 0x7fffffffu : ~order);
}

// A CTA's part of a row, in 16-byte vectors on the grid of the addresses: vector v holds the
// tokens v * kVec - shift and on, those outside the row as -inf.
template <typename T>
struct Slice {
  static constexpr int kVec = 16 / sizeof(T);
  const T* row;
  int V, shift, v0, v1;
  const uint4* held;  // of v0 and on, in shared memory, or null

  PE_DEV int token(int v) const { return v * kVec - shift; }
  PE_DEV uint4 load(int v) const {
    const int e = token(v);
    if (e >= 0 && e + kVec <= V) return ld_stream16(row + e);
    float f[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[i] = e + i >= 0 && e + i < V ? Elem<T>::to_f(row[e + i]) : -INFINITY;
    return pack16<T>(f);
  }
  PE_DEV uint4 get(int v) const { return held ? held[v - v0] : load(v); }
};

// Sum over the CTA, in a fixed order; all threads get it.
PE_DEV double cta_sum(double v, double* warps) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.;
  for (int w = 0; w < kWarps; ++w) s += warps[w];
  return s;
}

struct Cut {
  uint32_t key;   // order of the last kept token's logit
  int ties;       // kept ones with that logit, the first by index
  int all;        // all of them are kept
  double mass;    // weight of the kept ones
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  constexpr int kVec = 16 / sizeof(T);
  extern __shared__ uint4 held[];
  __shared__ Scratch sh;
  __shared__ Entry list[kList];     // on rank 0: the row's candidates
  __shared__ int mine_i[kList];     // this CTA's
  __shared__ float mine_x[kList];
  __shared__ uint32_t n_list, n_mine;
  __shared__ Best best_of[kMaxCluster];
  __shared__ uint32_t h_cnt[kBins], h_least[kBins];
  __shared__ unsigned long long h_mass[kBins];
  __shared__ double warp_d[kWarps];
  __shared__ float warp_m[kWarps], warp_lo[kWarps];
  __shared__ unsigned long long warp_k[kWarps];
  __shared__ int warp_i[kWarps];
  __shared__ float set_sh[4];
  __shared__ int req_sh;
  __shared__ uint32_t cut_sh[2];
  __shared__ int cut_count_sh, cut_n_sh;
  pdl_trigger();
  // (every CTA of the cluster has to have begun before another one writes to it)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  const int row = blockIdx.x / a.ctas, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = blockIdx.x - row * a.ctas, nr = a.ctas;
  Slice<T> s;
  s.row = static_cast<const T*>(a.logits) + row * a.ld;
  s.V = a.V;
  s.shift = static_cast<int>((reinterpret_cast<uintptr_t>(s.row) & 15u) / sizeof(T));
  {
    const int nvec = (a.V + s.shift + kVec - 1) / kVec, per = (nvec + nr - 1) / nr;
    s.v0 = min(static_cast<int>(rank) * per, nvec);
    s.v1 = min(s.v0 + per, nvec);
    s.held = nullptr;
  }
  // ---------------- settings
  if (warp == 0) {
    const int r = request_of(a.qsl, a.B, row, lane);
    if (lane == 0) {
      req_sh = r;
      uint32_t st = 0;
      if (r >= 0) {
        if (request_rows(a.qsl, r, a.T).bad) st |= PE_ST_ROWS_RANGE;
        const float t = a.temperature ? a.temperature[r] : 1.f;
        if (!(t >= 0.f)) st |= PE_ST_SAMPLING;
        const int k = a.top_k ? a.top_k[r] : 0;
        const float p = a.top_p ? a.top_p[r] : 1.f, mp = a.min_p ? a.min_p[r] : 0.f;
        if (p != p || mp != mp) st |= PE_ST_SAMPLING;
        set_sh[0] = temperature_of(t);
        set_sh[1] = __int_as_float(k <= 0 || k >= a.V ? 0 : k);
        set_sh[2] = p < 1.f ? p : 1.f;   // (NaN: 1)
        set_sh[3] = mp > 0.f ? mp : 0.f;  // (NaN: 0)
      }
      if (rank == 0 && st) set_status(a.status, st);
    }
  }
  if (tid < kBins) {
    h_cnt[tid] = 0;
    h_least[tid] = 0xffffffffu;
    h_mass[tid] = 0;
  }
  if (tid == 0) n_list = n_mine = 0;
  // ---------------- the slice, its largest logit
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  __syncthreads();
  if (req_sh < 0) return;  // (the whole cluster)
  float m = -INFINITY;
  for (int v = s.v0 + tid; v < s.v1; v += kUnroll * kThreads) {
    uint4 u[kUnroll];
#pragma unroll
    for (int x = 0; x < kUnroll; ++x)
      if (v + x * kThreads < s.v1) u[x] = s.load(v + x * kThreads);
#pragma unroll
    for (int x = 0; x < kUnroll; ++x)
      if (v + x * kThreads < s.v1) {
        m = max_nan(m, vec_max<T>(u[x]));
        if (a.resident) held[v + x * kThreads - s.v0] = u[x];
      }
  }
  if (a.resident) s.held = held;
  {
    float wm = m, lo = m > -INFINITY ? m : INFINITY;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      wm = max_nan(wm, __shfl_xor_sync(0xffffffffu, wm, o));
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
    if (lane == 0) {
      warp_m[warp] = wm;
      warp_lo[warp] = lo;
    }
    __syncthreads();
    if (warp == 0) {
      wm = lane < kWarps ? warp_m[lane] : -INFINITY;
      lo = lane < kWarps ? warp_lo[lane] : INFINITY;
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        wm = max_nan(wm, __shfl_xor_sync(0xffffffffu, wm, o));
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      }
      if (lane < nr) {
        put32(&sh.from[rank].m, lane, __float_as_uint(wm));
        put32(&sh.from[rank].lo, lane, __float_as_uint(lo));
      }
    }
  }
  row_sync();
  float M = -INFINITY, lo = INFINITY;
  for (uint32_t i = 0; i < nr; ++i) {
    M = max_nan(M, sh.from[i].m);
    lo = fminf(lo, sh.from[i].lo);
  }
  const float temp = set_sh[0], top_p = set_sh[2], min_p = set_sh[3];
  const int top_k = __float_as_int(set_sh[1]);

  // The CTA's best (order, index), and of the cluster; rank 0 writes the token.
  auto finish = [&](unsigned long long k, int i, bool cluster) {
    warp_best(k, i);
    if (lane == 0) {
      warp_k[warp] = k;
      warp_i[warp] = i;
    }
    __syncthreads();
    if (warp == 0) {
      k = lane < kWarps ? warp_k[lane] : 0ull;
      i = lane < kWarps ? warp_i[lane] : 0x7fffffff;
      warp_best(k, i);
      if (cluster && lane == 0) {
        put64(&best_of[rank].order, 0, k);
        put32(&best_of[rank].idx, 0, i);
      }
    }
    if (cluster) {
      row_sync();
      if (rank == 0 && warp == 0) {
        k = lane < nr ? best_of[lane].order : 0ull;
        i = lane < nr ? best_of[lane].idx : 0x7fffffff;
        warp_best(k, i);
      }
    }
    if (rank == 0 && tid == 0) {
      a.token[row] = k ? i : -1;
      if (!k) set_status(a.status, PE_ST_SAMPLING);
    }
  };

  // ---------------- greedy: the first token with the largest logit
  if (temp == 0.f) {
    int first = 0x7fffffff;
    if (m == M || M != M) {
      for (int v = s.v0 + tid; v < s.v1 && first == 0x7fffffff; v += kThreads) {
        float f[kVec];
        unpack16<T>(s.get(v), f);
#pragma unroll
        for (int e = kVec - 1; e >= 0; --e) {
          const int t = s.token(v) + e;
          if ((M != M ? f[e] != f[e] : f[e] == M) && t >= 0 && t < a.V) first = t;
        }
      }
    }
    finish(first < 0x7fffffff ? 1ull : 0ull, first, true);
    return;
  }
  if (!(fabsf(M) < INFINITY)) {  // no distribution
    if (rank == 0 && tid == 0) {
      a.token[row] = -1;
      set_status(a.status, PE_ST_SAMPLING);
    }
    return;
  }
  const float c = scale_of(temp), it = 1.f / temp;
  const float* noise = a.gumbel + row * a.ld_g;
  auto exact_score = [&](float x, float g) {
    return score_order((static_cast<double>(x) - static_cast<double>(M)) / static_cast<double>(temp) + g);
  };

  // Race over the slice's tokens that come no later than the cut (key 0: over all), with a
  // weight of at least min_p.  A thread keeps its best score in fp32; the threads whose best
  // is within reach of the CTA's (a score's rounding is 2^-23 of its two terms; noise past 128
  // is infinite) compare in 64 bits.
  auto race = [&](uint32_t key, bool all, int ties) {
    const bool wide = !((reinterpret_cast<uintptr_t>(noise) - s.shift * 4u) & 15u);
    float bs = -INFINITY, bx = 0.f, bg = 0.f;
    int bi = 0x7fffffff, seen = 0;  // seen: tokens at the cut before this trip's
    for (int vb = s.v0; vb < s.v1; vb += kThreads) {
      const int v = vb + tid;
      float f[kVec], g[kVec];
      int eq = 0;
      const int t0 = s.token(v);
      if (v < s.v1) {
        unpack16<T>(s.get(v), f);
        bool any = false;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const uint32_t o = argmax_order(f[e]);
          if (!all && o == key) ++eq;
          if (o < key || (min_p > 0.f && f[e] != M && ex2((f[e] - M) * c) < min_p)) f[e] = -INFINITY;
          any |= f[e] > -INFINITY;
        }
        if (any) {
          if (wide && t0 >= 0 && t0 + kVec <= a.V) {
#pragma unroll
            for (int e = 0; e < kVec; e += 4) unpack16<float>(ld_stream16(noise + t0 + e), g + e);
          } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) g[e] = f[e] > -INFINITY ? noise[t0 + e] : 0.f;
          }
        }
      }
      int place = 0;
      if (!all) {  // which of the equal ones are the first
        int incl = eq;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        __syncthreads();
        if (lane == 31) warp_i[warp] = incl;
        __syncthreads();
        place = seen + incl - eq;
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) place += warp_i[w];
          seen += warp_i[w];
        }
      }
      if (v < s.v1) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          if (!all && argmax_order(f[e]) == key && place++ >= ties) continue;
          const float sc = f[e] > -INFINITY ? fmaf(f[e] - M, it, g[e]) : -INFINITY;
          if (sc > bs) {
            bs = sc;
            bi = t0 + e;
            bx = f[e];
            bg = g[e];
          }
        }
      }
    }
    __syncthreads();
    const float wt = warp_max(bs);
    if (lane == 0) warp_m[warp] = wt;
    __syncthreads();
    float top = warp_m[0];
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, warp_m[w]);
    unsigned long long k = 0ull;
    if (bs > -INFINITY && (bs == top || bs >= top - 1e-6f * (fabsf(top) + fabsf(bs) + 128.f)))
      k = exact_score(bx, bg);
    else
      bi = 0x7fffffff;
    finish(k, bi, true);
  };

  const bool cut_k = top_k > 0, cut_p = top_p < 1.f;
  if (!cut_k && !cut_p && min_p == 0.f) {
    race(0u, true, 0);
    return;
  }

  // ---------------- a bound from below for the cut
  const float span = M - lo;
  const float scale = span > 0.f && span < INFINITY ? fminf(kBins / span, 1e30f) : 0.f;
  float bound = -INFINITY;
  double z_row = 0.;  // the weight of the whole row, where no top-k is set
  bool have_bound = false;
  if (cut_k || cut_p) {
    double z = 0.;
    if (!cut_k) {  // the weight of the whole row
      float z32 = 0.f;
      for (int v = s.v0 + tid; v < s.v1; v += kThreads) {
        float f[kVec], w = 0.f;
        unpack16<T>(s.get(v), f);
#pragma unroll
        for (int e = 0; e < kVec; ++e) w += ex2((f[e] - M) * c);
        z32 += w;
      }
      z = cta_sum(z32, warp_d);
    }
    if (m > -INFINITY) {
      const int b = min(kBins - 1, static_cast<int>((M - m) * scale));
      atomicAdd(&h_cnt[b], 1u);
      atomicMin(&h_least[b], argmax_order(m));
      if (!cut_k) atomicAdd(&h_mass[b], static_cast<unsigned long long>(ex2((m - M) * c) * 0x1p40f));
    }
    __syncthreads();
    for (uint32_t i = tid; i < kBins * nr; i += kThreads) {
      const uint32_t b = i % kBins, to = i / kBins;
      put32(&sh.from[rank].cnt[b], to, h_cnt[b]);
      put32(&sh.from[rank].least[b], to, h_least[b]);
      put64(&sh.from[rank].mass[b], to, h_mass[b]);
    }
    if (tid < nr) put64(&sh.from[rank].z, tid, __double_as_longlong(z));
    row_sync();
    for (uint32_t i = 0; i < nr; ++i) z_row += sh.from[i].z;
    if (warp == 0) {
      // (a margin for the roundings of the sums)
      const double need = cut_k ? static_cast<double>(top_k) : z_row * fmaxf(top_p, 0.f) * 1.000001;
      // two bins a lane
      double have[2];
      uint32_t least[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        unsigned long long q = 0;
        least[e] = 0xffffffffu;
        for (uint32_t i = 0; i < nr; ++i) {
          q += cut_k ? sh.from[i].cnt[2 * lane + e] : sh.from[i].mass[2 * lane + e];
          least[e] = min(least[e], sh.from[i].least[2 * lane + e]);
        }
        have[e] = cut_k ? static_cast<double>(q) : static_cast<double>(q) * 0x1p-40;
      }
      double before = have[0] + have[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      before -= have[0] + have[1];
      // the first bin with which there is enough
      const bool at0 = before + have[0] >= need, at1 = before + have[0] + have[1] >= need;
      const unsigned hit = __ballot_sync(0xffffffffu, at1);
      const int last = hit ? __ffs(hit) - 1 : 32;
      uint32_t o = 0xffffffffu;
      if (lane < last) o = min(least[0], least[1]);
      if (lane == last) o = at0 ? least[0] : min(least[0], least[1]);
      o = __reduce_min_sync(0xffffffffu, o);
      if (lane == 0) {
        cut_sh[0] = hit != 0 && o != 0xffffffffu;
        cut_sh[1] = o;
      }
    }
    __syncthreads();
    have_bound = cut_sh[0];
    if (have_bound) bound = logit_of(cut_sh[1]);
  } else {
    have_bound = true;  // min-p alone: the weights say it
  }

  // ---------------- the candidates
  if (have_bound) {
    const bool by_w = !cut_k && !cut_p;
    for (int v = s.v0 + tid; v < s.v1; v += kThreads) {
      const uint4 u = s.get(v);
      const float vm = vec_max<T>(u);
      if (by_w ? ex2((vm - M) * c) < min_p && vm != M : vm < bound) continue;
      float f[kVec];
      unpack16<T>(u, f);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const bool in = by_w ? f[e] == M || ex2((f[e] - M) * c) >= min_p : f[e] >= bound;
        if (in && f[e] > -INFINITY) {
          const uint32_t at = atomicAdd(&n_mine, 1u);
          if (at < kList) {
            mine_i[at] = s.token(v) + e;
            mine_x[at] = f[e];
          }
        }
      }
    }
    __syncthreads();
    const uint32_t n = n_mine;
    if (tid < nr) put32(&sh.from[rank].cand, tid, n);
    if (n <= kList) {
      __shared__ uint32_t start_sh;
      if (tid == 0) start_sh = n ? add32(&n_list, 0, n) : 0u;
      __syncthreads();
      const uint32_t at = start_sh + tid;
      if (tid < n && at < kList) {
        const int t = mine_i[tid];
        put64(&list[at].key, 0, argmax_key(mine_x[tid], static_cast<uint32_t>(t)));
        put32(&list[at].g, 0, __float_as_uint(noise[t]));
      }
    }
    row_sync();
    uint32_t total = 0;
    for (uint32_t i = 0; i < nr; ++i) total += min(static_cast<uint32_t>(sh.from[i].cand), kList + 1u);
    if (total <= kList) {
      if (rank != 0) return;
      // ---------------- rank and weight before each candidate
      unsigned long long key = 0ull, before = 0ull;
      int place = 0;
      float x = -INFINITY, w = 0.f, g = 0.f;
      if (tid < total) {
        key = list[tid].key;
        g = list[tid].g;
        x = logit_of(static_cast<uint32_t>(key >> 32));
        w = ex2((x - M) * c);
      }
      __shared__ unsigned long long q_sh[kList];
      const unsigned long long q = static_cast<unsigned long long>(w * 0x1p40f);
      q_sh[tid] = q;
      __syncthreads();
      if ((tid & ~31) < total) {
        for (uint32_t j = 0; j < total; ++j) {
          const bool ahead = list[j].key > key;
          place += ahead;
          before += ahead ? q_sh[j] : 0ull;
        }
      }
      bool keep = tid < total && (!cut_k || place < top_k);
      if (cut_p) {
        const double sum = cut_k ? cta_sum(keep ? static_cast<double>(q) : 0., warp_d) : z_row * 0x1p40;
        keep = keep && (place == 0 || static_cast<double>(before) < static_cast<double>(top_p) * sum);
      }
      keep = keep && (place == 0 || w >= min_p);
      finish(keep ? exact_score(x, g) : 0ull, static_cast<int>(~static_cast<uint32_t>(key)), false);
      return;
    }
  }

  // ---------------- the cut digit by digit
  // By all CTAs of the row alike: among the tokens whose order starts with the digits found so
  // far, counts and weights per next digit; the cut lies in the last digit with a kept token,
  // that is one with less than k tokens and less than `most` of weight before it.
  auto weight_bits = [&](float x) { return static_cast<uint32_t>(ex2((x - M) * c) * 0x1p31f); };
  auto descend = [&](int k, double frac, double z, int& my_ties) {
    uint32_t prefix = 0;
    unsigned long long count = 0, mass = 0;  // before the prefix
    unsigned long long n_eq = 0;
    double most = INFINITY;
    for (int level = 0; level < 4; ++level) {
      const int lshift = 24 - 8 * level;
      uint32_t (*h)[4] = sh.digits[level & 1];
      __syncthreads();
      for (int i = tid; i < kDigits * 4; i += kThreads) (&h[0][0])[i] = 0;
      __syncthreads();
      for (int v = s.v0 + tid; v < s.v1; v += kThreads) {
        float f[kVec];
        unpack16<T>(s.get(v), f);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const uint32_t o = argmax_order(f[e]);
          if (f[e] == -INFINITY || (level > 0 && o >> (lshift + 8) != prefix >> (lshift + 8))) continue;
          const uint32_t d = o >> lshift & 0xffu, q = weight_bits(f[e]);
          atomicAdd(&h[d][0], 1u);
          atomicAdd(&h[d][1], q & 0x7ffu);
          atomicAdd(&h[d][2], q >> 11 & 0x3ffu);
          atomicAdd(&h[d][3], q >> 21);
        }
      }
      row_sync();
      // the row's sums, from the largest digit down; thread t has digit 255 - t
      unsigned long long n_d = 0, m_d = 0;
      uint32_t own = 0;
      if (tid < kDigits) {
        const int d = kDigits - 1 - tid;
        own = h[d][0];
        for (uint32_t i = 0; i < nr; ++i) {
          n_d += get32(&h[d][0], i);
          m_d += get32(&h[d][1], i) + (static_cast<unsigned long long>(get32(&h[d][2], i)) << 11) +
                 (static_cast<unsigned long long>(get32(&h[d][3], i)) << 21);
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
      __shared__ unsigned long long scan_n[kWarps], scan_m[kWarps];
      if (lane == 31) {
        scan_n[warp] = ni;
        scan_m[warp] = mi;
      }
      if (tid == 0) cut_n_sh = -1;
      __syncthreads();
      unsigned long long cb = count + ni - n_d, mb = mass + mi - m_d, m_all = 0;
      for (int w = 0; w < kDigits / 32; ++w) {
        if (w < warp) {
          cb += scan_n[w];
          mb += scan_m[w];
        }
        m_all += scan_m[w];
      }
      // (the first token is kept whatever top_p is: nothing is before it)
      if (level == 0) most = frac >= 1. ? INFINITY : fmax(frac * (z >= 0. ? z : static_cast<double>(m_all)), 0.5);
      const bool in = tid < kDigits && n_d > 0 && cb < static_cast<unsigned long long>(k) && static_cast<double>(mb) < most;
      if (in) atomicMax(&cut_n_sh, tid);
      __syncthreads();
      if (tid == cut_n_sh) {
        cut_sh[0] = static_cast<uint32_t>(kDigits - 1 - tid);
        cut_sh[1] = own;
        scan_n[0] = cb;
        scan_m[0] = mb;
        scan_n[1] = n_d;
      }
      __syncthreads();
      prefix |= cut_sh[0] << lshift;
      my_ties = static_cast<int>(cut_sh[1]);
      count = scan_n[0];
      mass = scan_m[0];
      n_eq = scan_n[1];
    }
    Cut cut;
    cut.key = prefix;
    const uint32_t q = weight_bits(logit_of(prefix));
    double t = static_cast<double>(n_eq);
    t = fmin(t, static_cast<double>(k) - static_cast<double>(count));
    if (most < INFINITY && q > 0) t = fmin(t, ceil((most - static_cast<double>(mass)) / q));
    t = fmax(t, 1.);
    cut.ties = static_cast<int>(t);
    cut.all = t >= static_cast<double>(n_eq);
    cut.mass = static_cast<double>(mass) + t * q;
    return cut;
  };
  int ties = 0;
  Cut cut{0u, 0, 1, 0.};
  if (cut_k || cut_p) {
    const int k = cut_k ? top_k : 0x7fffffff;
    // top-p of what top-k leaves: the weight of that first
    double z = -1.;
    if (cut_k) {
      cut = descend(k, 1., -1., ties);
      z = cut.mass;
    }
    if (cut_p) cut = descend(k, static_cast<double>(top_p), z, ties);
    if (!cut.all) {
      // the CTAs' shares of the equal ones
      __syncthreads();
      if (tid == 0) cut_count_sh = ties;
      row_sync();
      int before = 0;
      for (uint32_t i = 0; i < rank; ++i) before += static_cast<int>(get32(&cut_count_sh, i));
      cut.ties = max(0, cut.ties - before);
    }
  }
  race(cut.key, cut.all, cut.ties);
  // (race ends behind a barrier of the cluster: no CTA reads another's memory after it)
}

// CTAs of a row, and whether its slices fit in their shared memory: few CTAs, as long as
// two of them fit on an SM, and more of them where the rows are too few for the SMs.
constexpr int kSliceTwo = 80 * 1024, kSliceOne = 176 * 1024;

struct Split {
  int ctas, resident;
  size_t smem;
};
Split split_of(int T, int V, int esize, int num_sms) {
  const int64_t bytes = static_cast<int64_t>(V) * esize + 32;
  int64_t n = std::min<int64_t>((bytes + kSliceTwo - 1) / kSliceTwo, kMaxCluster);
  while (n < kMaxCluster && static_cast<int64_t>(T) * (n + 1) <= 2 * num_sms && bytes / (n + 1) >= 8192) ++n;
  Split s;
  s.ctas = static_cast<int>(n);
  const int64_t vecs = (bytes / 16 + 1 + n - 1) / n;
  s.resident = vecs * 16 <= kSliceOne;
  s.smem = s.resident ? static_cast<size_t>(vecs * 16) : 0;
  return s;
}

template <typename T>
cudaError_t launch(const SampleArgs& a, size_t smem, cudaStream_t st) {
  // the function's shared-memory limit, once per device (a bit each; past 63 every time)
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (!(set.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSliceOne);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.T) * a.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[3];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
  attr[1].val.sharedMemCarveout = cudaSharedmemCarveoutMaxShared;
  attr[2].id = cudaLaunchAttributeClusterDimension;
  attr[2].val.clusterDim.x = a.ctas;
  attr[2].val.clusterDim.y = 1;
  attr[2].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 3;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
}

}  // namespace
}  // namespace pe

using namespace pe;

extern "C" size_t pe_sample_workspace_bytes(int max_batch, int max_rows, int vocab) {
  return max_batch < 0 || max_rows < 0 || vocab < 1 ? 0 : 256;
}

extern "C" int pe_sample(int B, int T, const int32_t* qsl, const void* logits, int64_t ld_logits, int vocab, int dtype,
                         const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                         const float* gumbel, int64_t ld_gumbel, int32_t* token, void* ws, size_t ws_bytes,
                         void* stream) {
  NvtxRange nvtx("pe_sample");
  if (B < 0 || T < 0 || vocab < 1 || ld_logits < vocab || ld_gumbel < vocab) return PE_ERR_ARG;
  if (dtype != PE_DTYPE_F32 && dtype != PE_DTYPE_BF16) return PE_ERR_UNSUPPORTED;
  if (B == 0) return T == 0 ? PE_OK : PE_ERR_ARG;
  if (B > 65535 || vocab > 1 << 24 || T > 0x7fffffff / kMaxCluster) return PE_ERR_UNSUPPORTED;
  if (!qsl || !ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < 256) return PE_ERR_ARG;
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
  a.status = static_cast<uint32_t*>(ws);
  const Split s = split_of(T, vocab, esize, sms);
  a.ctas = s.ctas;
  a.resident = s.resident;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == PE_DTYPE_F32 ? launch<float>(a, s.smem, st) : launch<bf16>(a, s.smem, st);
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}
