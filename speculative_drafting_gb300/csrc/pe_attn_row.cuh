// One row of chunk attention by a CTA of four warps, fp32 throughout: a warp takes every
// fourth group of 32 keys.  For the scores a lane owns a key (one reduction over the warp
// per group, not per key); for P V a lane owns every 32nd dimension.
#pragma once

#include "pe_common.cuh"
#include "pe_paged.h"

namespace pe {

constexpr int kRowWarps = 4;

struct RowScratch {
  __align__(16) float q[128];
  float m[kRowWarps], l[kRowWarps], acc[kRowWarps][128];
};

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

// The row's query, scaled; a barrier of the CTA has to follow.
template <typename T>
PE_DEV void row_query(const ChunkArgs& a, int row, int h, RowScratch& sh) {
  const T* q = static_cast<const T*>(a.q) + row * a.ld_q + static_cast<int64_t>(h) * a.hd;
  const int tid = threadIdx.x;
  if (tid < a.hd) sh.q[tid] = Elem<T>::to_f(q[tid]) / sqrtf(static_cast<float>(a.hd));
}

// Bits s .. s + 31 of a mask row of `words` words; those before bit 0 are set, those behind
// the last word are not.
PE_DEV uint32_t mask_bits(const uint32_t* bits, int words, int64_t s) {
  if (s <= -32) return 0xffffffffu;
  if (s >= 32ll * words) return 0u;
  const int w = static_cast<int>(s >> 5), sh = static_cast<int>(s & 31);  // w: -1 and on
  const uint32_t lo = w < 0 ? 0xffffffffu : bits[w], hi = w + 1 < words ? bits[w + 1] : 0u;
  return __funnelshift_r(lo, hi, sh);
}

// Keys 0 .. lim of request r for its row `row` (of all), head h; of a tree (kTree), of the keys
// from `first` on those whose bit is set in the row's mask.
template <typename T, bool kTree>
PE_DEV void attend_row(const ChunkArgs& a, const TreeMask& mask, int r, int row, int h, int lim, int first,
                       RowScratch& sh) {
  constexpr int kVec = 16 / sizeof(T);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = h / (a.H / a.G);
  const T* kc = static_cast<const T*>(a.k_cache);
  const T* vc = static_cast<const T*>(a.v_cache);
  float m = -INFINITY, l = 0.f;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t t0 = 32 * warp; t0 <= lim; t0 += 32 * kRowWarps) {
    // scores: this lane's key
    const int t = static_cast<int>(t0) + lane;
    int64_t base = -1;
    float s = -INFINITY;
    if (t0 + lane <= lim && (!kTree || t0 + 31 < first ||
                             (mask_bits(mask.bits + static_cast<int64_t>(row) * mask.words, mask.words, t0 - first) >> lane & 1u))) {
      const int blk = a.block_table[static_cast<int64_t>(r) * a.max_blocks + t / a.bs];
      if (blk < 0 || blk >= a.num_blocks) {
        set_status(a.status, PE_ST_BLOCK_RANGE);
      } else {
        base = ((static_cast<int64_t>(blk) * a.G + g) * a.bs + t % a.bs) * a.hd;
        const uint4* k = reinterpret_cast<const uint4*>(kc + base);
        s = 0.f;
#pragma unroll 4
        for (int i = 0; i < a.hd / kVec; ++i) s = dot16<T>(k[i], sh.q + i * kVec, s);
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
    sh.m[warp] = m;
    sh.l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < a.hd) sh.acc[warp][lane + 32 * i] = acc[i];
  __syncthreads();
  // a sink logit joins the maximum and the denominator (its value row is zero); a warp
  // that saw no key has l = 0 (NaN: it saw one)
  const float sk = a.sink ? a.sink[h] : -INFINITY;
  float M = sk;
  for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, sh.m[w]);
  auto weight = [&](int w) { return sh.l[w] == 0.f ? 0.f : sh.m[w] == -INFINITY ? sh.l[w] : expf(sh.m[w] - M); };
  float den = sk == -INFINITY ? 0.f : expf(sk - M);
  bool any = false;
  for (int w = 0; w < kRowWarps; ++w) {
    den += weight(w) * sh.l[w];
    any |= sh.l[w] != 0.f;
  }
  T* out = static_cast<T*>(a.out) + row * a.ld_out + static_cast<int64_t>(h) * a.hd;
  for (int d = tid; d < a.hd; d += 32 * kRowWarps) {
    float num = 0.f;
    for (int w = 0; w < kRowWarps; ++w) num += weight(w) * sh.acc[w][d];
    out[d] = Elem<T>::from_f(any ? num / den : 0.f);
  }
}

}  // namespace pe
