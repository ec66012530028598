// What the calls that draw tokens share (pe_verify_sampled, pe_sample).
#pragma once

#include "pe_common.cuh"

namespace pe {

// a temperature as it is used
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
PE_DEV int request_of(const int32_t* qsl, int B, int row, int lane) {
  int lo = 0, hi = B;  // qsl[lo] <= row < qsl[hi], were qsl[B] past every row
  if (qsl[B] <= row || qsl[0] > row) return -1;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < hi && qsl[min(at, B)] <= row);
    const int k = 31 - __clz(le | 1u);
    const int nlo = lo + k * step;
    hi = min(hi, nlo + step);
    lo = nlo;
  }
  return lo;
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

}  // namespace pe
