// Attention of each request's new rows over its pages on the tensor cores (bf16,
// head size 64 or 128, blocks of a multiple of 8 keys).
//
//   S = Q K^T, P = exp(S / sqrt(hd) - m), l = sum P, O = P V, out = O / l
//
// in one pass over tiles of 128 keys (head size 64) or 64 (128) with a running maximum m
// per row; S, P and O live in tensor memory, K and V come by TMA, page by page.
//
// The rows of a request that share a KV head (n_r tokens x H/G heads, token-major)
// are cut into units of up to 256 rows.  One CTA works on one unit at a time with
// two streams of 128 rows, each with softmax warps of its own, so that one stream's
// products run while the other's exponentials do:
//   wide unit   (129..256 rows): stream s holds rows 128 s ..; both read every tile;
//   narrow unit (at most 128 rows: verify rows, single tokens): both streams hold
//               the same rows and take the tiles in turn; their (m, l, O) join at
//               the end through tensor memory.
//
// Work split.  The units of all KV heads form one line, each as long as its cost
// (rows in use x keys, plus a constant); CTA c takes the c-th of equal pieces, cut
// at tiles.  A unit cut between CTAs leaves unnormalised partials (m, l, O) in the
// workspace, at most two per CTA, and a second kernel joins them.  Every CTA finds
// its piece itself from qsl and seq_len, so the host needs no lengths.
//
// Infinities and NaN.  A key that some rows of a unit see and others do not has weight 0
// in the others' product, and 0 times what is not finite is NaN.  Rows whose result is
// not finite though their l is a number, in units with a value that is not finite past
// some row's last key, are computed again by the second kernel from the keys that they see.
//
// Trees.  Every unit goes over all of its request's keys.  Tiles of the context alone are as
// without a tree; in the others a thread takes its row's bits of the tile's keys out of the mask
// while the product runs.  64 requests of 1 to 64 nodes over 512 to 8192 keys, 8 query heads a KV
// head of 64: 242 us, of which the bytes would take 86 and the operations 73.  Issue slots are used
// 51 % of the time and the tensor pipe 35 %: the steps of a tile wait for one another, as in a
// prompt.  Requests of more than 32 nodes read their keys once for each unit (826 MB for 581).
//
// Warps: 0-7 softmax of stream 0 (two warps to 32 rows, half the keys of a tile each),
// 8-15 of stream 1, 16 K tiles and the unit list, 17 and 18 the products of either stream,
// 19 V tiles.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <type_traits>

#include "pe_attn_row.cuh"
#include "pe_tmem.cuh"

namespace pe {
namespace {

constexpr int kThreads = 640;     // four softmax warpgroups, one of K, V and product warps
constexpr int kRows = 128;        // rows per stream
constexpr int kUnitRows = 256;
constexpr int kItems = 4;         // unit descriptors in flight
constexpr int kMasks = 16;        // tile masks in flight
constexpr float kLog2e = 1.4426950408889634f;
// The running maximum is raised only when a row's new one is more than 2^8 above
// it: O is rarely rescaled.  P is at most 2^8, so O of values below 2^120 / keys stays
// finite; the sums round relatively, whatever the scale.
constexpr float kLazy = 8.f;

template <int HD>
struct Shape {
  static constexpr int kHalves = HD / 64;             // 128-byte columns of a row
  static constexpr int kTile = HD == 64 ? 128 : 64;   // keys per tile
  static constexpr int kTileBytes = kTile * HD * 2;   // a K or V tile
  static constexpr int kQBytes = kRows * HD * 2;      // a Q tile
  // bytes from one group of 8 keys of a K or V tile to the next (load_box)
  static constexpr int kGroupBytes = 1024 * kHalves;
  // slots of the K ring, and of the V ring: 128 KB in all
  static constexpr int kSlots = 4;
  // Q of a unit, and where its results pass through; with a second one the next unit's Q
  // and first S are on their way while this one's results are written
  static constexpr int kQBufs = HD == 64 ? 2 : 1;
  static constexpr int kSmem = 2 * kQBufs * kQBytes + 2 * kSlots * kTileBytes + 1024;
  // Tensor memory, 512 columns: S, P and O of two streams.  Head size 64: 128 + 64 + 64
  // columns each; S is free again once it is in registers.  Head size 128 leaves 128 for S
  // and P: two S buffers of a 64-key tile that the steps take in turn, with P in the
  // place of its S, free after P V.  (With one S of 128 keys, the next product waiting for
  // P V, the softmax warps waited for S two fifths of their time: mixed chunks 534 us,
  // 478 like this.)
  static constexpr bool kOverlay = HD == 128;
  static constexpr uint32_t kS = 0, kP = kOverlay ? 0 : 256, kPStride = kOverlay ? 128 : 64;
  static constexpr uint32_t kO = HD == 64 ? 384 : 256;
};

struct Req {
  int q0, n, L, R, Q;
  long long A;
};

// A place on the line of units: tile `tile` of unit `qt` of request r, KV head g.
struct Place {
  int g, r, qt, tile;
};

struct Unit {
  int r, g, q0, n, L;   // request, KV head, first row, rows, keys
  int row0, rows, wide; // first packed row, packed rows (1..256)
  int tile0, tile1;     // key tiles of this CTA's part
  int kend;             // keys any row of the unit sees
  int whole;            // the part is the whole unit
  int index;            // in this CTA's list
};

// What a CTA leaves for the second kernel.
struct Rec {
  int head;                  // its first unit began elsewhere: 1, and ends there too: 2
  int tail;                  // its last unit goes on in the next CTA: that unit's
  int q0, g, row0, rows, r;  // first row, KV head, packed rows, request
  int bad0, bad1;            // range of its whole units with rows to compute again
  int u_g, u_r, u_qt;        // where its list of units starts
  int pad[4];
};

struct TcArgs {
  ChunkArgs c;
  int box;          // keys per TMA box
  int grid;
  int hg_shift;     // H / G = 1 << hg_shift, -1 if it is no power of two
  int umin;         // least cost of a CTA's piece, in 128-key tiles of a narrow unit
  int overhead;     // constant cost of a unit, in the same measure
  float* part_o;    // [grid][2][part_rows][hd]
  float* part_ml;   // [grid][2][part_rows][2]
  int part_rows;
  Rec* rec;         // [grid]
};
struct TcTreeArgs : TcArgs {
  TreeMask mask;
};
template <bool kTree>
using Args = std::conditional_t<kTree, TcTreeArgs, TcArgs>;
template <bool kTree>
PE_DEV TreeMask mask_of(const Args<kTree>& p) {
  if constexpr (kTree) return p.mask;
  return TreeMask{};
}

template <bool kTree>
PE_DEV Req load_req(const ChunkArgs& a, int r, bool report) {
  const RowRange x = request_rows(a.qsl, r, a.T);
  Req q;
  q.q0 = x.q0;
  q.n = x.q1 - x.q0;
  const long long Lmax = static_cast<long long>(a.max_blocks) * a.bs;
  const int L = a.seq_len[r];
  const bool over = L < 0 || L > Lmax;
  q.L = over ? static_cast<int>(min(max(static_cast<long long>(L), 0ll), Lmax)) : L;
  if (report && (x.bad || over))
    set_status(a.status, (x.bad ? PE_ST_ROWS_RANGE : 0u) | (over ? PE_ST_BLOCK_RANGE : 0u));
  const int HG = a.H / a.G;
  q.R = q.n * HG;
  q.Q = (q.R + kUnitRows - 1) / kUnitRows;
  q.A = static_cast<long long>(kTree ? q.L : max(q.L - q.n, 0)) * HG;
  return q;
}

// keys that some row of unit i sees (of a tree: may see), and their tiles (at least one)
template <bool kTree>
PE_DEV int unit_kend(const Req& q, int i, int HG) {
  if (kTree) return q.L;
  const int last = (min((i + 1) * kUnitRows, q.R) - 1) / HG;
  return min(max(q.L - q.n + last + 1, 0), q.L);
}
template <int HD>
PE_DEV int unit_tiles(int kend) {
  return max(1, (kend + Shape<HD>::kTile - 1) / Shape<HD>::kTile);
}

// cost of unit i, and of the units before it (all but the last are wide; every row of a tree
// goes over all keys)
template <bool kTree>
PE_DEV long long unit_cost(const Req& q, int i, long long ov) {
  const int end = min((i + 1) * kUnitRows, q.R);
  return (end - i * kUnitRows > kRows ? 2 : 1) * (q.A + (kTree ? 0 : end)) + ov;
}
template <bool kTree>
PE_DEV long long units_before(const Req& q, int i, long long ov) {
  return i * (2 * q.A + ov) + (kTree ? 0 : 256ll * i * (i + 1));
}
template <bool kTree>
PE_DEV long long req_cost(const Req& q, long long ov) {
  return q.Q == 0 ? 0 : units_before<kTree>(q, q.Q - 1, ov) + unit_cost<kTree>(q, q.Q - 1, ov);
}

// the first request at or after r that has rows (B if none), by one whole warp
PE_DEV int next_request(const ChunkArgs& a, int r, int lane) {
  for (; r < a.B; r += 32) {
    int n = 0;
    if (r + lane < a.B) {
      const RowRange x = request_rows(a.qsl, r + lane, a.T);
      n = x.q1 - x.q0;
    }
    const unsigned any = __ballot_sync(0xffffffffu, n > 0);
    if (any) return r + __ffs(any) - 1;
  }
  return a.B;
}

PE_DEV uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// One box of keys: rows `row` .. of the cache.  Head size 64: [keys][128 bytes].  Head
// size 128: both 128-byte halves of 8 keys at a time, [keys / 8][half][8][128 bytes], so
// that one copy brings whole rows (a copy per half took twice the TMA's time).
template <int HD>
PE_DEV void load_box(void* dst, const CUtensorMap* map, uint64_t* bar, int row, uint64_t policy) {
  if (HD == 64) {
    tma_load_2d(dst, map, bar, 0, row, policy);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::"
        "cache_hint [%0], [%1, {%3, %3, %3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(row >> 3), "l"(policy)
        : "memory");
  }
}

// One lane of a whole warp, the same one every time.
PE_DEV bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

// `zero`, with NaN in it if one of the eight values is not finite
PE_DEV __nv_bfloat162 not_finite(const uint4& v, __nv_bfloat162 zero) {
  const __nv_bfloat162 none = __float2bfloat162_rn(0.f);
  zero = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.x), none, zero);
  zero = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.y), none, zero);
  zero = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.z), none, zero);
  return __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.w), none, zero);
}

// packed row -> token, head in the group
PE_DEV void split_row(const TcArgs& p, int row, int& tok, int& head) {
  const int HG = p.c.H / p.c.G;
  tok = p.hg_shift >= 0 ? row >> p.hg_shift : row / HG;
  head = row - tok * HG;
}

// Places of a softmax thread: stream s, half hf of the keys and columns, rows 32 wq ..
struct Seat {
  int lane, s, hf, wq, i;
};
PE_DEV Seat seat_of(int tid) {
  Seat t;
  t.lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  t.s = warp >> 3;
  t.hf = warp >> 2 & 1;
  t.wq = warp & 3;
  t.i = t.wq * 32 + t.lane;
  return t;
}
// 16-byte chunk ch of a row of a Q tile, 128-byte swizzle
PE_DEV uint4* tile_at(uint8_t* tile, int row, int ch) {
  return reinterpret_cast<uint4*>(tile + (ch >> 3) * (kRows * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
}
template <int HD>
PE_DEV uint8_t* q_tile(uint8_t* q_sm, const Unit& u, int tile) {
  return q_sm + ((Shape<HD>::kQBufs == 2 ? (u.index & 1) * 2 : 0) + tile) * Shape<HD>::kQBytes;
}
// Half rows move between global and shared memory kLpr lanes to a row: each instruction
// covers kRpi rows of a warp's 32.
template <int HD>
struct Lines {
  static constexpr int kLpr = HD / 16, kRpi = 32 / kLpr;
};

// What softmax warps do between units is in calls that are not inlined, with rolled loops:
// it is cold code (unrolled, its instruction fetches cost 5000 clocks a unit at head size
// 64, 12000 at 128), and inlined, what it needs stays in registers through the steps and
// pushes others out of them (prompt of 8192: 695 us, 64 x 8 rows 125 us).

// A unit's Q on its way to shared memory, or to L2.
template <int HD>
PE_DEV void load_q(const TcArgs& p, const Unit& u, uint8_t* q_sm, bool to_l2) {
  constexpr int kLpr = Lines<HD>::kLpr, kRpi = Lines<HD>::kRpi;
  const Seat t = seat_of(threadIdx.x);
  if (!u.wide && t.s != 0) return;
  const int HG = p.c.H / p.c.G, rel = u.wide ? t.s * kRows + t.i : t.i;
  const bool ok = rel < u.rows;
  int tok, head;
  split_row(p, u.row0 + (ok ? rel : 0), tok, head);
  const long long off = (u.q0 + tok) * p.c.ld_q + static_cast<long long>(u.g * HG + head) * HD;
  if (to_l2) {
    if (ok) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const bf16*>(p.c.q) + off + HD / 2 * t.hf));
    return;
  }
  const unsigned oks = __ballot_sync(0xffffffffu, ok);
  uint8_t* tile = q_tile<HD>(q_sm, u, u.wide ? t.s : 0);
#pragma unroll 2
  for (int it = 0; it < kLpr; ++it) {
    const int src = it * kRpi + t.lane / kLpr, ch = t.hf * kLpr + t.lane % kLpr;
    const long long o = __shfl_sync(0xffffffffu, off, src);
    cp_async16(smem_u32(tile_at(tile, t.wq * 32 + src, ch)), static_cast<const bf16*>(p.c.q) + o + ch * 8,
               oks >> src & 1);
  }
  cp_async_commit();
}

// A unit's results: through its Q tiles (whole units), or as fp32 partials straight to the
// workspace.  m and l are this thread's row's; those of a narrow unit's two streams join
// here, in stream 0's warps.  A whole unit is noted in bad if a value is not finite though
// its row's l is a number.  (One for the kernels with a tree, one for those without: a call that both
// share costs a prompt of 8192 573 us, 568 like this.)
template <int HD, bool kTree>
__device__ __noinline__ void finish_unit(const TcArgs& p, const Unit& u, int* bad, uint8_t* q_sm, uint32_t tmem,
                                         const float (*ml)[kRows][2], float m, float l) {
  constexpr int kLpr = Lines<HD>::kLpr, kRpi = Lines<HD>::kRpi;
  const ChunkArgs& a = p.c;
  const Seat t = seat_of(threadIdx.x);
  const bool wide = u.wide, whole = u.whole;
  const int rel = wide ? t.s * kRows + t.i : t.i;
  // (a whole warp's answer, and known as such: what follows is .aligned)
  if (__shfl_sync(0xffffffffu, (!wide && t.s != 0) || (rel & ~31) >= u.rows, 0)) return;
  const bool row_ok = rel < u.rows;
  int tok, head;
  split_row(p, u.row0 + (row_ok ? rel : 0), tok, head);
  head += u.g * (a.H / a.G);
  const size_t prow = (static_cast<size_t>(blockIdx.x) * 2 + (u.tile0 > 0 ? 0 : 1)) * p.part_rows + rel;
  float w0 = 1.f, w1 = 0.f;
  if (!wide) {
    const float m0 = ml[0][t.i][0], m1 = ml[1][t.i][0];
    m = fmaxf(m0, m1);
    w0 = m0 == -INFINITY ? 0.f : ex2(m0 - m);
    w1 = m1 == -INFINITY ? 0.f : ex2(m1 - m);
    l = ml[0][t.i][1] * w0 + ml[1][t.i][1] * w1;
  }
  if (!whole && row_ok && t.hf == 0) *reinterpret_cast<float2*>(p.part_ml + prow * 2) = make_float2(m, l);
  // factor of the unnormalised O of a whole unit: a sink joins m and l
  float f = 1.f;
  if (whole) {
    const float sk = a.sink && row_ok ? a.sink[head] * kLog2e : -INFINITY;
    const float top = fmaxf(m, sk);
    const float e = ex2(m - top);
    f = top == -INFINITY || l == 0.f ? 0.f : e / (l * e + (sk == -INFINITY ? 0.f : ex2(sk - top)));
  }
  const uint32_t tO = tmem + (static_cast<uint32_t>(t.wq * 32) << 16) + Shape<HD>::kO + (HD / 2) * t.hf;
  uint8_t* tile = q_tile<HD>(q_sm, u, t.s);
  const bool both = !wide && u.tile1 - u.tile0 > 1;
#pragma unroll 1
  for (int b = 0; b < HD / 32; ++b) {
    uint32_t o[16];
    tmem_ld16_issue(tO + (wide ? t.s * HD : 0) + 16 * b, o);
    tmem_wait_ld();
    tmem_use16(o);
    if (both) {
      uint32_t o1[16];
      tmem_ld16_issue(tO + HD + 16 * b, o1);
      tmem_wait_ld();
      tmem_use16(o1);
#pragma unroll
      for (int c = 0; c < 16; ++c)
        o[c] = __float_as_uint(__uint_as_float(o[c]) * w0 + __uint_as_float(o1[c]) * w1);
    }
    const int col = HD / 2 * t.hf + 16 * b;
    if (whole) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = pack_bf16x2(__uint_as_float(o[8 * c + 2 * e]) * f, __uint_as_float(o[8 * c + 2 * e + 1]) * f);
        *tile_at(tile, t.i, col / 8 + c) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else if (row_ok) {
      uint4* d = reinterpret_cast<uint4*>(p.part_o + prow * HD + col);
#pragma unroll
      for (int c = 0; c < 4; ++c) d[c] = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
    }
  }
  if (!whole) return;
  __syncwarp();
  const long long off = (u.q0 + tok) * a.ld_out + static_cast<long long>(head) * HD;
  bf16* out = static_cast<bf16*>(a.out);
  const unsigned oks = __ballot_sync(0xffffffffu, row_ok), nums = __ballot_sync(0xffffffffu, l == l);
  __nv_bfloat162 zero = __float2bfloat162_rn(0.f);  // NaN once a value is not finite
#pragma unroll 2
  for (int it = 0; it < kLpr; ++it) {
    const int src = it * kRpi + t.lane / kLpr, ch = t.hf * kLpr + t.lane % kLpr;
    const long long o = __shfl_sync(0xffffffffu, off, src);
    if (oks >> src & 1) {
      const uint4 v = *tile_at(tile, t.wq * 32 + src, ch);
      *reinterpret_cast<uint4*>(out + o + ch * 8) = v;
      if (nums >> src & 1) zero = not_finite(v, zero);
    }
  }
  if (__any_sync(0xffffffffu, __hisnan(zero.x) || __hisnan(zero.y)) && t.lane == 0) {
    atomicMin(&bad[0], u.index);
    atomicMax(&bad[1], u.index);
  }
  __syncwarp();
}

template <int HD, bool kTree>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_tc_kernel(const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Args<kTree> p) {
  using S = Shape<HD>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t k_full[S::kSlots], k_empty[S::kSlots];
  __shared__ __align__(8) uint64_t v_full[S::kSlots], v_empty[S::kSlots];
  __shared__ __align__(8) uint64_t it_full[kItems], it_empty[kItems];
  __shared__ __align__(8) uint64_t q_full[kItems][2], s_full[2][2], s_free[2], p_full[2], pv_done[2];
  __shared__ __align__(8) uint64_t x_bar[2];
  __shared__ __align__(8) uint64_t end_bar;
  __shared__ Unit items[kItems];
  __shared__ uint32_t mask_sh[kMasks];  // per tile: bit j = keys 8j..8j+7 were loaded
  __shared__ float ml_sh[2][kRows][2];
  __shared__ float pair_sh[2][2][2][kRows];  // [stream][half][buffer][row]
  __shared__ long long scan_sh[kThreads / 32];
  __shared__ Place place_sh[2];
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  __shared__ Rec rec_sh;
  __shared__ int bad_sh[2];  // first and last unit of the list with rows to compute again
  constexpr uint32_t kAll = (1u << S::kTile / 8) - 1;  // every group of 8 keys of a tile
  const ChunkArgs& a = p.c;
  // (values that are the same across a warp go through a shuffle: the compiler then
  // keeps them in the warp's uniform registers)
  auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  uint8_t* q_sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* k_ring = q_sm + 2 * S::kQBufs * S::kQBytes;
  uint8_t* v_ring = k_ring + S::kSlots * S::kTileBytes;
  const int HG = a.H / a.G;

  if (tid == 0) {
    // (a stalled slot's barrier expects an arrival that no one makes)
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&k_full[i], a.stall == 1 + i ? 2 : 1);
      mbar_init(&k_empty[i], 2);
      mbar_init(&v_full[i], a.stall == 1 + S::kSlots + i ? 2 : 1);
      mbar_init(&v_empty[i], 2);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], 16 + 3);
      mbar_init(&q_full[i][0], 8);
      mbar_init(&q_full[i][1], 8);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s][0], 1);
      mbar_init(&s_full[s][1], 1);
      mbar_init(&s_free[s], 8);
      mbar_init(&p_full[s], 8);
      mbar_init(&pv_done[s], 1);
      mbar_init(&x_bar[s], 16);
    }
    mbar_init(&end_bar, 2);
    abort_sh = 0;
    rec_sh.head = rec_sh.tail = 0;
    rec_sh.bad1 = -1;
    bad_sh[0] = INT_MAX;
    bad_sh[1] = -1;
    fence_barrier_init();
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  // tensor memory before the next kernel may start: a successor's CTA that held
  // some of it while waiting for this grid would keep this one from starting
  if (warp == 17) {
    tmem_alloc(&tmem_sh, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  pdl_trigger();
  pdl_wait();

  // ---------------- this CTA's piece of the line
  const long long ov = static_cast<long long>(p.overhead) * 128 * HG;
  const int per = (a.B + kThreads - 1) / kThreads;  // requests per thread
  const int r_lo = min(tid * per, a.B), r_hi = min(r_lo + per, a.B);
  long long mine = 0;
  Req req0;  // of this thread's first request (with up to kThreads requests, its only one)
  for (int r = r_lo; r < r_hi; ++r) {
    const Req q = load_req<kTree>(a, r, blockIdx.x == 0);
    if (kTree && blockIdx.x == 0 && q.n > 32 * mask_of<kTree>(p).words) set_status(a.status, PE_ST_TREE);
    if (r == r_lo) req0 = q;
    mine += req_cost<kTree>(q, ov);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) scan_sh[warp] = incl;
  if (tid < 2) place_sh[tid] = Place{a.G, 0, 0, 0};  // the end of the line
  __syncthreads();
  long long before = incl - mine, Wg = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scan_sh[w];
    Wg += scan_sh[w];
  }
  // Where the pieces begin is a matter of balance: fp32 serves (64-bit divisions cost a
  // small call a microsecond), so long as neighbours find the same place.  Every KV head
  // has the same line, so a whole number of pieces each: the nearest one where there are
  // CTAs to spare (one token over 2048 keys of 8 KV heads: 19 us, 22 us with pieces across
  // heads), else the next below unless that idles more than one CTA in 16.
  const long long W = Wg * a.G;
  const float least = static_cast<float>(p.umin * 128 * HG);
  int pieces = static_cast<int>(fminf(fmaxf(static_cast<float>(W) / least, 1.f), static_cast<float>(p.grid)));
  const bool spare = pieces < p.grid;
  const int per_head = spare ? min((pieces + a.G / 2) / a.G, p.grid / a.G) : pieces / a.G;
  const bool even = per_head > 0 && (spare || (pieces - per_head * a.G) * 16 <= pieces);
  if (even) pieces = per_head * a.G;
  // the first cost of piece c on its head's line: never past the line, no less for a
  // larger c
  auto piece = [&](int c, int& g) {
    if (even) {
      g = c / per_head;
      return static_cast<long long>(static_cast<float>(Wg) *
                                    (static_cast<float>(c - g * per_head) / static_cast<float>(per_head)));
    }
    long long w =
        static_cast<long long>(static_cast<float>(W) * (static_cast<float>(c) / static_cast<float>(pieces)));
    w = min(w, W - 1);
    g = min(a.G - 1, static_cast<int>(static_cast<float>(w) / static_cast<float>(Wg)));
    while (w < g * Wg) --g;
    while (w >= (g + 1) * Wg) ++g;
    return w - g * Wg;
  };
  const bool idle = W == 0 || static_cast<int>(blockIdx.x) >= pieces;
  if (!idle) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int c = blockIdx.x + e;
      if (c >= pieces) continue;  // the end of the line
      int g;
      long long rem = min(piece(c, g), Wg - 1) - before;
      if (rem < 0 || rem >= mine) continue;
      for (int r = r_lo; r < r_hi; ++r) {
        const Req q = r == r_lo ? req0 : load_req<kTree>(a, r, false);
        const long long cost = req_cost<kTree>(q, ov);
        if (rem >= cost) {
          rem -= cost;
          continue;
        }
        int lo = 0, hi = q.Q;  // the last unit that starts at or before rem
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (units_before<kTree>(q, mid, ov) <= rem) lo = mid; else hi = mid;
        }
        const long long off = rem - units_before<kTree>(q, lo, ov);
        const int kt = unit_tiles<HD>(unit_kend<kTree>(q, lo, HG));
        // A cut near a unit's end or start moves there: a part costs a CTA some tiles of
        // time whatever its length.
        const float cost_u = static_cast<float>(unit_cost<kTree>(q, lo, ov));
        const float len = static_cast<float>(W) / static_cast<float>(pieces) * static_cast<float>(kt) / cost_u;
        const int snap = min(4, static_cast<int>(0.25f * len));
        int tile = min(kt - 1, static_cast<int>(static_cast<float>(off) / cost_u * static_cast<float>(kt)));
        if (tile <= snap && 2 * tile < kt)
          tile = 0;
        else if (kt - tile <= snap)
          tile = kt;  // (no tile of this unit)
        place_sh[e] = Place{g, r, lo, tile};
        break;
      }
    }
  }
  __syncthreads();

  // columns from the first S (and P) to those of a stream's n-th step
  auto buffer = [](uint32_t n) { return S::kOverlay ? (n & 1) * S::kTile : 0u; };

  volatile int* abort_flag = &abort_sh;
  auto fail = [&]() {
    abort_sh = 1;
    set_status(a.status, PE_ST_TIMEOUT);
  };

  // the whole warp goes on or gives up together (what follows is .aligned)
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag)) != 0;
  };

  // The tiles of a unit's part into a ring, by one whole warp.  A window is 32 boxes (32 /
  // gpt tiles), one per lane; the block ids of the next window are read while the
  // current one streams.
  auto stream_tiles = [&](const Unit& u, bool is_v, uint8_t* ring, const CUtensorMap* map, uint64_t* full,
                          uint64_t* empty, uint32_t& loads) {
    const uint64_t policy = u.wide ? policy_evict_normal() : policy_evict_first();
    const int gpt = S::kTile / p.box;  // boxes per tile
    auto block_of = [&](int wn) {
      const long long key = (static_cast<long long>(wn) * 32 + lane) * p.box;
      return key < u.kend ? a.block_table[static_cast<long long>(u.r) * a.max_blocks + key / a.bs]
                          : -2;  // past the unit's keys
    };
    auto row_of = [&](int wn, int blk) {
      if (blk >= 0 && blk < a.num_blocks)
        return (blk * a.G + u.g) * a.bs + (wn * 32 + lane) * p.box % a.bs;
      if (blk != -2 || (wn * 32ll + lane) * p.box < u.kend) set_status(a.status, PE_ST_BLOCK_RANGE);
      return -1;
    };
    int wn = u.tile0 * gpt >> 5;
    int row = row_of(wn, block_of(wn)), next = block_of(wn + 1);
#pragma unroll 1
    for (int t = u.tile0; t < u.tile1; ++t, ++loads) {
      if (t * gpt >> 5 != wn) {
        ++wn;
        row = row_of(wn, next);
        next = block_of(wn + 1);
      }
      const int b0 = t * gpt & 31;
      const bool mine = lane >= b0 && lane < b0 + gpt && row >= 0;
      const unsigned have = __ballot_sync(0xffffffffu, mine);
      const int st = loads % S::kSlots;
      if (loads >= S::kSlots && !wait_warp(&empty[st], (loads / S::kSlots - 1) & 1)) return false;
      const int n = __popc(have);
      if (lane == 0) {
        if (!is_v) {
          uint32_t m = kAll;  // the boxes' bits, widened to groups of 8 keys
          if (n < gpt) {
            m = 0;
            const int w8 = p.box / 8;
            for (int b = 0; b < gpt; ++b)
              if (have >> (b0 + b) & 1) m |= ((1u << w8) - 1u) << (b * w8);
          }
          mask_sh[loads % kMasks] = m;
        }
        mbar_arrive_expect_tx(&full[st], n * p.box * HD * 2);
      }
      __syncwarp();
      if (mine)
        load_box<HD>(ring + st * S::kTileBytes + (lane - b0) * p.box * HD * 2, map, &full[st], row, policy);
    }
    return true;
  };
  // no copy may be in flight when the CTA leaves (after a timeout some may be)
  auto drain = [&](uint64_t* full, uint32_t loads) {
    int never = 0;
    for (uint32_t i = loads > S::kSlots ? loads - S::kSlots : 0; i < loads; ++i)
      mbar_wait(&full[i % S::kSlots], (i / S::kSlots) & 1, &never);
  };

  if (idle) {
    if (tid == 0) {
      p.rec[blockIdx.x].head = p.rec[blockIdx.x].tail = 0;
      p.rec[blockIdx.x].bad1 = -1;
    }
  } else if (warp < 16) {
    // registers: 640 x 96 at launch = 4 x 128 x 104 + 128 x 64
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // ---------------- softmax warpgroups: two threads per row, of two warps that share
    // the tensor-memory lanes; thread hf has half hf of a tile's keys and half the columns
    // of O.  (One thread per row left a scheduler two warps, in which the waits of a step
    // took longer than its exponentials.)
    const int s = warp >> 3, hf = warp >> 2 & 1, wq = warp & 3, i = wq * 32 + lane;
    const uint32_t tm = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    constexpr int kKeys = S::kTile / 2;  // this thread's of a tile
    const uint32_t tS0 = tm + S::kS + s * 128 + kKeys * hf, tP0 = tm + S::kP + s * S::kPStride + kKeys / 2 * hf;
    const uint32_t tO = tm + S::kO + (HD / 2) * hf;  // of stream 0; stream 1's HD columns on
    const float sc = kLog2e / sqrtf(static_cast<float>(HD));
    uint32_t n_items = 0, n_st = 0, tiles = 0, n_x = 0, n_pair = 0;
    bool failed = false;
    // One arrival for the warp, of all that its lanes did before.
    auto warp_arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // The two warps of a row meet at named barriers: a vote, and a value of this row from
    // the thread with its other half.  These have no time limit, so each warp comes to every
    // one that the other comes to: a warp whose wait gave up (`failed`) goes on without
    // waits to the end of the unit, where the two leave together.
    const int pair = 1 + s * 4 + wq;
    auto vote = [&](bool v) {
      uint32_t r;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\t"
          "setp.ne.u32 p, %1, 0;\n\t"
          "barrier.cta.red.or.pred.aligned q, %2, 64, p;\n\t"
          "selp.u32 %0, 1, 0, q;\n\t}\n"
          : "=r"(r)
          : "r"(static_cast<uint32_t>(v)), "r"(pair)
          : "memory");
      return __any_sync(0xffffffffu, r) != 0;  // (known to be the whole warp's)
    };
    auto partner = [&](float v) {
      const int buf = n_pair++ & 1;
      pair_sh[s][hf][buf][i] = v;
      asm volatile("barrier.cta.sync.aligned %0, 64;" ::"r"(pair) : "memory");
      return pair_sh[s][hf ^ 1][buf][i];
    };
    // A unit's description stays in its slot until the unit is done: what the results
    // need of it is read again then, not held in registers through the steps.
    int cur = -1;  // slot of the unit at hand, -1: none is left
    // A unit's Q is there.  Both groups complete both Q barriers of the slot in every unit,
    // before they let go of it: an MMA warp that skips units (none of their tiles is its
    // stream's) finds the barriers in step.
    auto q_there = [&](int slot) {
      cp_async_wait<0>();
      fence_proxy_async();
      warp_arrive(&q_full[slot][s]);
    };
    // the next unit
    auto next_unit = [&]() {
      const int slot = n_items % kItems;
      if (!wait_warp(&it_full[slot], (n_items / kItems) & 1)) return false;
      ++n_items;
      cur = uniform(items[slot].r < 0 ? -1 : slot);
      return true;
    };
    failed = !next_unit();
    if (vote(failed)) {
      if (failed) fail();
      cur = -1;
    }
    while (cur >= 0) {
      const int slot = cur;
      const int nt = uniform(items[slot].tile1 - items[slot].tile0);
      const bool wide = uniform(items[slot].wide);
      const int rel = wide ? s * kRows + i : i;           // row within the unit
      const bool row_ok = rel < items[slot].rows;
      const bool live = uniform((rel & ~31) < items[slot].rows);  // some row of this warp exists
      const int kend = uniform(items[slot].kend), tile0 = uniform(items[slot].tile0);
      // the last key that this row sees, and the unit's first row (of a tree: its row of the
      // mask, and the context's last key)
      int lim, lim0;
      {
        int tok, head;
        split_row(p, items[slot].row0 + rel, tok, head);
        const int p0 = items[slot].L - items[slot].n;
        if constexpr (kTree) {
          lim = row_ok ? items[slot].q0 + tok : -1;
          lim0 = uniform(p0 - 1);
        } else {
          lim = row_ok ? p0 + tok : -1;
          split_row(p, items[slot].row0, tok, head);
          lim0 = uniform(p0 + tok);
        }
      }
      if (S::kQBufs == 1 || items[slot].index == 0) {
        load_q<HD>(p, items[slot], q_sm, false);
        q_there(slot);
      }
      const int mysteps = wide ? nt : (nt - s + 1) >> 1;
      float m = -INFINITY, l = 0.f;  // m: running maximum in units of log2
      for (int k = 0; k < mysteps; ++k) {
        const int j = wide ? k : 2 * k + s;
        const int t0 = (tile0 + j) * S::kTile;
        // (two S products of the overlay may be done before the first is looked at: a
        // barrier for either buffer)
        const uint32_t n = n_st + k;
        // (on their way while the product runs)
        uint32_t tree[kTree ? kKeys / 32 : 1];
        if constexpr (kTree) {
          if (t0 + S::kTile - 1 > lim0) {
#pragma unroll
            for (int b = 0; b < kKeys / 32; ++b)
              tree[b] = lim < 0 ? 0u
                                : mask_bits(p.mask.bits + static_cast<int64_t>(lim) * p.mask.words, p.mask.words,
                                            t0 + kKeys * hf + 32 * b - static_cast<int64_t>(lim0 + 1));
          } else {
#pragma unroll
            for (int b = 0; b < kKeys / 32; ++b) tree[b] = lim < 0 ? 0u : 0xffffffffu;
          }
        }
        failed = failed || !wait_warp(&s_full[s][S::kOverlay ? n & 1 : 0], (S::kOverlay ? n >> 1 : n) & 1);
        tc_fence_after();
        const uint32_t have = uniform(mask_sh[(tiles + j) % kMasks]);
        const bool inner = t0 + S::kTile - 1 <= lim0 && have == kAll;
        uint32_t x[kKeys];
        const int c0 = t0 + kKeys * hf;
        const uint32_t tS = tS0 + buffer(n), tP = tP0 + buffer(n);
        float best = -INFINITY;  // this row's largest score of the tile
        if (live) {
          if (inner) {
            uint32_t mx[kKeys / 32];
#pragma unroll
            for (int b = 0; b < kKeys / 32; ++b) tmem_ld32_max_issue(tS + 32 * b, x + 32 * b, mx[b]);
            tmem_wait_ld();
#pragma unroll
            for (int b = 0; b < kKeys / 32; ++b) {
              tmem_use32(x + 32 * b);
              tmem_use(mx[b]);
              best = fmaxf(best, __uint_as_float(mx[b]));
            }
          } else {
#pragma unroll
            for (int b = 0; b < kKeys / 32; ++b) tmem_ld32_issue(tS + 32 * b, x + 32 * b);
            tmem_wait_ld();
#pragma unroll
            for (int b = 0; b < kKeys / 32; ++b) tmem_use32(x + 32 * b);
            const uint32_t mine = have >> (kKeys / 8 * hf);
            if constexpr (kTree) {
#pragma unroll
              for (int b = 0; b < kKeys / 32; ++b) {
                // this row's keys of 32: in its mask, there, before the request's end
                uint32_t see = tree[b];
                const int left = kend - c0 - 32 * b;
                if (left < 32) see &= left <= 0 ? 0u : (1u << left) - 1u;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (!(mine >> (4 * b + e) & 1u)) see &= ~(0xffu << 8 * e);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                  if (!(see >> c & 1u)) x[32 * b + c] = 0xff800000u;
                  best = fmaxf(best, __uint_as_float(x[32 * b + c]));
                }
              }
            } else {
#pragma unroll
              for (int c = 0; c < kKeys; ++c) {
                if (c0 + c > lim || !(mine >> (c >> 3) & 1u)) x[c] = 0xff800000u;
                best = fmaxf(best, __uint_as_float(x[c]));
              }
            }
          }
        }
        if (!S::kOverlay) {
          tc_fence_before();
          warp_arrive(&s_free[s]);
        }
        if (live) {
          // raise the maximum: at the first finite score, or when it climbed far
          best *= sc;
          if (vote(best > m + kLazy || (m == -INFINITY && best > m))) {
            const float top = fmaxf(best, partner(best));
            const bool raise = top > m + kLazy || (m == -INFINITY && top > m);
            const float mn = raise ? top : m;
            const float f = (m == -INFINITY) ? 1.f : ex2(m - mn);
            m = mn;
            l *= f;
            if (k > 0) {
              failed = failed || !wait_warp(&pv_done[s], (n_st + k - 1) & 1);
              tc_fence_after();
#pragma unroll 1
              for (int b = 0; b < HD / 32; ++b) {
                uint32_t o[16];
                tmem_ld16_issue(tO + s * HD + 16 * b, o);
                tmem_wait_ld();
                tmem_use16(o);
#pragma unroll
                for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                tmem_st16_issue(tO + s * HD + 16 * b, o);
              }
              tmem_wait_st();
            }
          }
          const float off = m == -INFINITY ? 0.f : m;
          const uint64_t sc2 = pack_f32x2(sc, sc), off2 = pack_f32x2(-off, -off);
          uint64_t ls = 0ull;
#pragma unroll
          for (int c = 0; c < kKeys; c += 2) {
            float p0, p1;
            unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sc2, off2),
                         p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            ls = add_f32x2(ls, pack_f32x2(p0, p1));
            // P enters the product as bf16 (relative 2^-8 at most, the size of the
            // result's own rounding); the sum l takes the unrounded weights.  (Low parts in a
            // second product, in units of at most 128 rows only: error against 64 bits 0.0023
            // -> 0.0017, 64 x 8 rows 110 -> 187 us, one token 17.2 -> 19.4, 32K 610 -> 642.
            // Tensor memory is full at head size 64: the low parts take S's place.)
            x[c >> 1] = pack_bf16x2(p0, p1);
          }
          float l0, l1;
          unpack_f32x2(ls, l0, l1);
          l += l0 + l1;
        }
        // the last P V of this stream has read P (and, with the overlay, the product warp
        // has taken the p_full before this one)
        if (k > 0) failed = failed || !wait_warp(&pv_done[s], (n_st + k - 1) & 1);
        if (live) {
          tc_fence_after();
          if constexpr (kKeys == 64)
            tmem_st32_issue(tP, x);
          else
            tmem_st16_issue(tP, x);
          tmem_wait_st();
        }
        // Keys that no row sees (past the unit's last, or of a skipped block) hold
        // anything, NaN included: their V rows become 0 before the product
        const bool cut = t0 + S::kTile > kend || have != kAll;
        if (cut) {
          const uint32_t idx = tiles + j;
          failed = failed || !wait_warp(&v_full[idx % S::kSlots], (idx / S::kSlots) & 1);
          if (!failed && i < S::kTile && (t0 + i >= kend || !(have >> (i >> 3) & 1u))) {
            uint8_t* v = v_ring + (idx % S::kSlots) * S::kTileBytes + (i >> 3) * S::kGroupBytes + (i & 7) * 128;
#pragma unroll
            for (int c = 0; c < HD / 16; ++c) {
              const int ch = hf * (HD / 16) + c;
              *reinterpret_cast<uint4*>(v + (ch >> 3) * 1024 + ((ch & 7) << 4)) = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async();
        }
        tc_fence_before();
        warp_arrive(&p_full[s]);
      }
      // the next unit's Q, then the last P V of this one
      failed = failed || !next_unit();
      if (!failed && cur >= 0) load_q<HD>(p, items[cur], q_sm, S::kQBufs == 1);
      if (mysteps > 0) failed = failed || !wait_warp(&pv_done[s], (n_st + mysteps - 1) & 1);
      if (S::kQBufs == 2 && !failed && cur >= 0) q_there(cur);
      n_st += mysteps;
      tiles += nt;
      tc_fence_after();
      if (live) l += partner(l);
      // the two streams' states of a narrow unit's rows join in stream 0's warps
      if (!wide) {
        if (hf == 0) {
          ml_sh[s][i][0] = m;
          ml_sh[s][i][1] = l;
        }
        tc_fence_before();
        warp_arrive(&x_bar[0]);
        failed = failed || !wait_warp(&x_bar[0], n_x & 1);
        tc_fence_after();
      }
      if (!failed) finish_unit<HD, kTree>(p, items[slot], bad_sh, q_sm, tmem, ml_sh, m, l);
      tc_fence_before();
      if (!wide) {
        // stream 1's O and ml_sh have been read
        warp_arrive(&x_bar[1]);
        failed = failed || !wait_warp(&x_bar[1], n_x & 1);
        ++n_x;
      }
      if (vote(failed)) {
        if (failed) fail();
        cp_async_wait<0>();  // no copy of Q is in flight when the CTA leaves
        break;
      }
      warp_arrive(&it_empty[slot]);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 16) {
    // ---------------- K warp: lists the units of this CTA's piece and streams their K
    // tiles (the V warp, below, their V tiles: one warp issues a 2 KB box every 90 ns,
    // half of what an SM's share of DRAM needs at head size 64)
    const Place first = place_sh[0], last = place_sh[1];
    Place cur = first;
    uint32_t loads = 0, n_items = 0;
    bool go = true;
    Req q;
    int q_of = -1;
    while (go) {
      if (cur.g > last.g || (cur.g == last.g && (cur.r > last.r || (cur.r == last.r && cur.qt > last.qt))))
        break;
      const bool ends_here = cur.g == last.g && cur.r == last.r && cur.qt == last.qt;
      if (ends_here && last.tile <= cur.tile) break;
      if (cur.g >= a.G) break;
      if (cur.r != q_of) {
        q = load_req<kTree>(a, cur.r, false);
        q_of = cur.r;
      }
      Unit u;
      u.r = cur.r;
      u.g = cur.g;
      u.q0 = q.q0;
      u.n = q.n;
      u.L = q.L;
      u.row0 = cur.qt * kUnitRows;
      u.rows = min(kUnitRows, q.R - u.row0);
      u.wide = u.rows > kRows;
      u.kend = unit_kend<kTree>(q, cur.qt, HG);
      const int kt = unit_tiles<HD>(u.kend);
      u.tile0 = cur.tile;
      u.tile1 = ends_here ? min(last.tile, kt) : kt;
      u.index = static_cast<int>(n_items);
      const bool some = u.tile0 < u.tile1;
      u.whole = u.tile0 == 0 && u.tile1 == kt;
      if (some && !u.whole && lane == 0) {
        if (u.tile0 > 0) {
          rec_sh.head = u.tile1 == kt ? 2 : 1;
        } else {
          rec_sh.tail = 1;
          rec_sh.q0 = u.q0;
          rec_sh.g = u.g;
          rec_sh.row0 = u.row0;
          rec_sh.rows = u.rows;
          rec_sh.r = u.r;
        }
      }
      if (some) {
      // hand the unit over
      const int slot = n_items % kItems;
      if (n_items >= kItems) {
        int ok = lane == 0 ? mbar_wait(&it_empty[slot], (n_items / kItems - 1) & 1, abort_flag) : 1;
        if (!__shfl_sync(0xffffffffu, ok, 0)) {
          if (lane == 0) fail();
          go = false;
          break;
        }
      }
      if (lane == 0) {
        items[slot] = u;
        mbar_arrive(&it_full[slot]);
      }
      if (n_items == 0 && lane == 0) {
        rec_sh.u_g = u.g;
        rec_sh.u_r = u.r;
        rec_sh.u_qt = cur.qt;
      }
      ++n_items;
      if (!stream_tiles(u, false, k_ring, &kmap, k_full, k_empty, loads)) {
        fail();
        go = false;
      }
      }
      // the next unit
      if (ends_here) break;
      cur.tile = 0;
      if (++cur.qt >= q.Q) {
        cur.qt = 0;
        cur.r = next_request(a, cur.r + 1, lane);
        if (cur.r >= a.B) {
          ++cur.g;
          cur.r = next_request(a, 0, lane);
        }
      }
    }
    // the end of the list
    if (lane == 0) {
      const int slot = n_items % kItems;
      if (n_items < kItems || mbar_wait(&it_empty[slot], (n_items / kItems - 1) & 1, abort_flag)) {
        items[slot].r = -1;
        items[slot].rows = items[slot].wide = items[slot].row0 = 0;
        mbar_arrive(&it_full[slot]);
      }
      p.rec[blockIdx.x] = rec_sh;
    }
    drain(k_full, loads);
    __syncwarp();
    } else if (warp == 19) {
    // ---------------- V warp
    uint32_t loads = 0;
    for (uint32_t n_items = 0;; ++n_items) {
      const int slot = n_items % kItems;
      if (!wait_warp(&it_full[slot], (n_items / kItems) & 1)) {
        fail();
        break;
      }
      const Unit u = items[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&it_empty[slot]);
      if (u.r < 0) break;
      if (!stream_tiles(u, true, v_ring, &vmap, v_full, v_empty, loads)) {
        fail();
        break;
      }
    }
    drain(v_full, loads);
    __syncwarp();
    } else {
    // ---------------- MMA warps, one per stream: the waits of one overlap the products
    // of the other (a single warp for both took 1436 clocks a tile of head size 64, in
    // which the tensor pipe worked 614).  All lanes follow the steps and an elected one
    // issues: in a branch of one lane the operands' descriptors go through vector
    // registers for every product (955 clocks a tile against 690 in isolation).
    const int s = warp - 17;
    uint32_t tiles = 0, seen_k = 0, seen_v = 0, n_items = 0, n_st = 0;
    const uint32_t idesc_s = idesc_bf16_f32(kRows, S::kTile);
    const uint32_t idesc_o = idesc_bf16_f32(kRows, HD) | (1u << 16);  // V is MN-major
    const uint32_t dS = tmem + S::kS + s * 128, dP = tmem + S::kP + s * S::kPStride;
    const uint32_t dO = tmem + S::kO + s * HD;
    // the stride between groups of 8 keys, past the 1024 bytes of the descriptors' default
    constexpr uint64_t kWider = static_cast<uint64_t>((S::kGroupBytes - 1024) / 16) << 32;
    constexpr int kOwn = 2;  // this stream's S products ahead of its P V
    bool go = true;
    while (go) {
      const int slot = n_items % kItems;
      if (!wait_warp(&it_full[slot], (n_items / kItems) & 1)) {
        fail();
        break;
      }
      const Unit u = items[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&it_empty[slot]);
      ++n_items;
      if (u.r < 0) break;
      const int nt = u.tile1 - u.tile0;
      const int steps = u.wide ? nt : (nt - s + 1) >> 1;     // of this stream
      const int qb = u.wide ? s : 0, q_at = S::kQBufs == 2 ? (u.index & 1) * 2 + qb : qb;
      // (with no step here the other stream may run units ahead: nothing to wait for)
      if (steps > 0) go = wait_warp(&q_full[slot][qb], ((n_items - 1) / kItems) & 1);
      const uint64_t ad = sw128_kmajor_desc(smem_u32(q_sm + q_at * S::kQBytes));
      // Both warps see every load of both rings in order, the other stream's too: a
      // slot's barrier then never is a phase behind or ahead of the one that is waited
      // for.  A slot is free when both have let go of it, its users once their products
      // are done.
      auto take = [&](uint64_t* full, uint64_t* empty, uint32_t& seen, uint32_t to) {
        for (; seen < to; ++seen) {
          if (!wait_warp(&full[seen % S::kSlots], (seen / S::kSlots) & 1)) return false;
          if (elect_one()) mbar_arrive(&empty[seen % S::kSlots]);
        }
        return true;
      };
      auto wait_load = [&](uint64_t* full, uint64_t* empty, uint32_t& seen, uint32_t idx) {
        if (!take(full, empty, seen, idx)) return false;
        ++seen;
        return wait_warp(&full[idx % S::kSlots], (idx / S::kSlots) & 1);
      };
#pragma unroll 1
      for (int k = -kOwn; k < steps && go; ++k) {
        if (k >= 0) {  // O += P V of step k
          const int j = u.wide ? k : 2 * k + s;
          const uint32_t idx = tiles + j;
          const int st = idx % S::kSlots;
          go = wait_load(v_full, v_empty, seen_v, idx) && wait_warp(&p_full[s], (n_st + k) & 1);
          if (!go) break;
          tc_fence_after();
          // column blocks of 64 lie 1024 bytes apart, groups of 8 keys kGroupBytes
          const uint64_t bd = sw128_mnmajor_desc(smem_u32(v_ring + st * S::kTileBytes), 1024) + kWider;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < S::kTile / 16; ++kk)
              umma_bf16_ta(dO, dP + buffer(n_st + k) + kk * 8, bd + kk * (2 * S::kGroupBytes / 16), idesc_o,
                           k > 0 || kk > 0);
            umma_commit(&pv_done[s]);
            umma_commit(&v_empty[st]);
          }
          // with the overlay P's place is that of the next S but one (or of the next unit's
          // second S, whose Q may come from the other stream's warps)
          if (S::kOverlay) go = wait_warp(&pv_done[s], (n_st + k) & 1);
          if (!go) break;
        }
        const int n = k + kOwn;
        if (n < steps) {  // S = Q K^T of step n
          const int j = u.wide ? n : 2 * n + s;
          const uint32_t idx = tiles + j;
          const int st = idx % S::kSlots;
          go = wait_load(k_full, k_empty, seen_k, idx);
          // the S of the step before is in registers (the unit before's is)
          if (go && !S::kOverlay && n > 0) go = wait_warp(&s_free[s], (n_st + n - 1) & 1);
          if (!go) break;
          tc_fence_after();
          const uint64_t bd = sw128_kmajor_desc(smem_u32(k_ring + st * S::kTileBytes)) + kWider;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
              const uint32_t in = (kk & 3) * 2, half = kk >> 2;
              umma_bf16(dS + buffer(n_st + n), ad + half * (kRows * 128 / 16) + in,
                        bd + half * (1024 / 16) + in, idesc_s, kk > 0);
            }
            umma_commit(&s_full[s][S::kOverlay ? (n_st + n) & 1 : 0]);
            umma_commit(&k_empty[st]);
          }
        }
      }
      tiles += nt;
      if (!go || !take(k_full, k_empty, seen_k, tiles) || !take(v_full, v_empty, seen_v, tiles)) {
        fail();
        break;
      }
      n_st += steps;
    }
    // nothing of this warp is running when the CTA leaves
    int never = 0;
    if (elect_one()) umma_commit(&end_bar);
    mbar_wait(&end_bar, 0, &never);
    __syncwarp();
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && bad_sh[1] >= 0) {
    p.rec[blockIdx.x].bad0 = bad_sh[0];
    p.rec[blockIdx.x].bad1 = bad_sh[1];
  }
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

PE_DEV bool finite(float v) { return fabsf(v) <= FLT_MAX; }

// The i-th row of a unit for this warp of the join (its slice: blockIdx.y)
PE_DEV int join_row(int i, int warp) { return (blockIdx.y + i * gridDim.y) * kRowWarps + warp; }

// Of the unit at packed row row0, the rows noted (bit i of a warp's `again`: its i-th row),
// so far as a key of the unit is past them.  (This and the next one are calls, not inlined:
// their registers would be the join's.)
template <bool kTree>
__device__ __noinline__ void redo_unit(const Args<kTree>& p, int r, int g, int row0, uint32_t again,
                                       RowScratch& scratch) {
  __shared__ uint32_t again_sh[kRowWarps];
  const ChunkArgs& a = p.c;
  const int HG = a.H / a.G;
  if ((threadIdx.x & 31) == 0) again_sh[threadIdx.x >> 5] = again;
  __syncthreads();
  const Req q = load_req<kTree>(a, r, false);
  const int kend = unit_kend<kTree>(q, row0 / kUnitRows, HG);
  // Only where a value that some row does not see (at most the unit's tokens) is not finite:
  // what all of its rows see reached them rightly.
  const int t0 = max(kTree ? q.L - q.n : q.L - q.n + row0 / HG + 1, 0), chunks = a.hd / 8;
  __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
  for (int i = threadIdx.x; i < (kend - t0) * chunks; i += 32 * kRowWarps) {
    const int t = t0 + i / chunks;
    const int blk = a.block_table[static_cast<long long>(r) * a.max_blocks + t / a.bs];
    if (blk < 0 || blk >= a.num_blocks) continue;
    const long long key = (static_cast<long long>(blk) * a.G + g) * a.bs + t % a.bs;
    zero = not_finite(reinterpret_cast<const uint4*>(a.v_cache)[key * chunks + i % chunks], zero);
  }
  if (!__syncthreads_or(__hisnan(zero.x) || __hisnan(zero.y))) return;
  for (int w = 0; w < kRowWarps; ++w)
    for (uint32_t todo = again_sh[w]; todo; todo &= todo - 1) {
      const int row = row0 + join_row(__ffs(todo) - 1, w);
      const int tok = row / HG, head = g * HG + row % HG, lim = kTree ? q.L - 1 : q.L - q.n + tok;
      if (!kTree && lim >= kend - 1) continue;
      row_query<bf16>(a, q.q0 + tok, head, scratch);
      __syncthreads();
      attend_row<bf16, kTree>(a, mask_of<kTree>(p), r, q.q0 + tok, head, lim, q.L - q.n, scratch);
      __syncthreads();
    }
  __syncthreads();
}

// The whole units of this CTA's list up to the last that was noted, as the K warp of the
// first kernel went through them.
template <int HD, bool kTree>
__device__ __noinline__ void redo_list(const Args<kTree>& p, RowScratch& scratch) {
  const ChunkArgs& a = p.c;
  const Rec& rec = p.rec[blockIdx.x];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, HG = a.H / a.G;
  const int bad0 = rec.bad0, bad1 = rec.bad1;
  int g = rec.u_g, r = rec.u_r, qt = rec.u_qt;
  for (int unit = 0; unit <= bad1; ++unit) {
    const Req q = load_req<kTree>(a, r, false);
    if (unit >= bad0) {
      const int n = min(kUnitRows, q.R - qt * kUnitRows);
      uint32_t again = 0;
      for (int at = 0, row; (row = join_row(at, warp)) < n; ++at) {
        const int tok = (qt * kUnitRows + row) / HG, head = g * HG + (qt * kUnitRows + row) % HG;
        const bf16* o =
            static_cast<const bf16*>(a.out) + (q.q0 + tok) * a.ld_out + static_cast<long long>(head) * HD;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < HD / 32; ++i) bad |= !finite(__bfloat162float(o[lane + 32 * i]));
        again |= static_cast<uint32_t>(__any_sync(0xffffffffu, bad)) << at;
      }
      redo_unit<kTree>(p, r, g, qt * kUnitRows, again, scratch);
    }
    if (++qt >= q.Q) {
      qt = 0;
      r = next_request(a, r + 1, lane);
      if (r >= a.B) {
        ++g;
        r = next_request(a, 0, lane);
      }
    }
  }
}

// Joins the partials of the units that were cut between CTAs.  CTA (c, y): the unit
// whose first part is CTA c's last one, a slice of its rows; its other parts are the
// first ones of the CTAs after c, up to the one that ends it.  One warp per row.  Then the
// rows to compute again: of that unit, and of CTA c's whole units that have some.
template <int HD, bool kTree>
__global__ void __launch_bounds__(32 * kRowWarps) chunk_join_kernel(const __grid_constant__ Args<kTree> p) {
  constexpr int V = HD / 32;
  __shared__ RowScratch scratch;
  pdl_trigger();
  pdl_wait();
  const ChunkArgs& a = p.c;
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Rec& rec = p.rec[c];
  const int bad1 = rec.bad1;
  if (!rec.tail && bad1 < 0) return;
  const int HG = a.H / a.G;
  uint32_t again = 0;  // the rows of this warp to compute again
  // (the same for every row)
  const int code0 = c + lane >= p.grid ? 0 : lane == 0 ? 1 : p.rec[c + lane].head;
  const int q0 = rec.q0, g = rec.g, row0 = rec.row0, rows = rec.tail ? rec.rows : 0;
  // (m, l) of a row in the part of CTA k, its `head` being code
  auto load_ml = [&](int k, int code, bool part, int row) {
    const size_t prow = (static_cast<size_t>(k) * 2 + (k == c)) * p.part_rows + row;
    return part && code != 0 && row < rows ? *reinterpret_cast<const float2*>(p.part_ml + prow * 2)
                                           : make_float2(-INFINITY, 0.f);
  };
  // the next row's, of the first 32 CTAs, is on its way while a row is joined
  const unsigned ends0 = __ballot_sync(0xffffffffu, code0 == 2 || c + lane >= p.grid);
  const bool in0 = lane <= (ends0 ? __ffs(ends0) - 1 : 31);
  float2 ahead = load_ml(c + lane, code0, in0, join_row(0, warp));
  for (int at = 0, row; (row = join_row(at, warp)) < rows; ++at) {
    const float2 ml0 = ahead;
    ahead = load_ml(c + lane, code0, in0, join_row(at + 1, warp));
    const int tok = (row0 + row) / HG, head = g * HG + (row0 + row) % HG;
    float M = a.sink ? a.sink[head] * kLog2e : -INFINITY;  // the sink: one more part, O = 0
    float den = M == -INFINITY ? 0.f : 1.f;
    bool any = false;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    // 32 CTAs at a time, a lane each: which of them hold a part, and its (m, l)
    bool more = true;
    for (int k0 = c; more; k0 += 32) {
      const int k = k0 + lane;
      const int code = k0 == c ? code0 : k >= p.grid ? 0 : p.rec[k].head;
      const unsigned ends = __ballot_sync(0xffffffffu, code == 2 || k >= p.grid);
      const int last = ends ? __ffs(ends) - 1 : 31;  // of this window
      more = !ends;
      const bool part = code != 0 && lane <= last;
      const float2 ml = k0 == c ? ml0 : load_ml(k, code, part, row);
      // (l = 0: no key of the part was seen; NaN counts as seen)
      const bool seen = ml.y != 0.f;
      any |= __any_sync(0xffffffffu, seen);
      const float mn = fmaxf(M, warp_max(ml.x));
      const float keep = M == -INFINITY ? 0.f : ex2(M - mn);
      const float w = !seen ? 0.f : ml.x == -INFINITY ? ml.y : ex2(ml.x - mn);
      M = mn;
      den = den * keep + warp_sum(w * ml.y);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] *= keep;
      unsigned todo = __ballot_sync(0xffffffffu, part && seen);
      while (todo) {
        // four parts' loads in flight, added in order
        float o[4][V], wj[4];
        int n = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int j = todo ? __ffs(todo) - 1 : 0;
          wj[x] = __shfl_sync(0xffffffffu, w, j);
          const bool ok = todo != 0;
          todo &= todo - 1;
          n += ok;
          const float* src =
              p.part_o + ((static_cast<size_t>(k0 + j) * 2 + (k0 + j == c)) * p.part_rows + row) * HD;
#pragma unroll
          for (int i = 0; i < V; ++i) o[x][i] = ok ? src[lane + 32 * i] : 0.f;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (x < n)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] += wj[x] * o[x][i];
      }
    }
    const float inv = any ? 1.f / den : 0.f;
    bf16* out = static_cast<bf16*>(a.out) + (q0 + tok) * a.ld_out + static_cast<long long>(head) * HD;
#pragma unroll
    for (int i = 0; i < V; ++i) out[lane + 32 * i] = __float2bfloat16_rn(acc[i] * inv);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < V; ++i) bad |= !finite(acc[i]);
    again |= static_cast<uint32_t>(__any_sync(0xffffffffu, bad && den == den)) << at;
  }
  if (__syncthreads_or(again)) redo_unit<kTree>(p, rec.r, g, row0, again, scratch);
  if (bad1 >= 0) redo_list<HD, kTree>(p, scratch);
}

constexpr int kMaxGrid = 152;

size_t al256(size_t x) { return (x + 255) / 256 * 256; }

int part_rows_of(int T, int HG) {
  return static_cast<long long>(T) * HG > kRows ? kUnitRows : kRows;
}

// offsets past the 256-byte header: records, (m, l), O
size_t rec_bytes() { return al256(kMaxGrid * sizeof(Rec)); }
size_t ml_bytes(int part_rows) { return al256(size_t{kMaxGrid} * 2 * part_rows * 2 * sizeof(float)); }

template <int HD, bool kTree>
int launch(const Args<kTree>& p, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  // the function's shared-memory limit, once per device (a bit each; past 63 every time)
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PE_ERR_CUDA;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (!(set.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(chunk_tc_kernel<HD, kTree>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Shape<HD>::kSmem) != cudaSuccess)
      return PE_ERR_CUDA;
    set.fetch_or(bit, std::memory_order_release);
  }
  if (launch_chained(chunk_tc_kernel<HD, kTree>, dim3(p.grid), dim3(kThreads), Shape<HD>::kSmem, st, km, vm, p) !=
      cudaSuccess)
    return PE_ERR_CUDA;
  // Rows of a unit per warp of the join (it notes them in 32 bits).  A warp's rows wait for one another; with
  // fewer for each the grid has as many more CTAs, most of which find no cut unit.  So 8 CTAs of 4 warps to
  // a unit of as many rows as one can have (one token 18.6 -> 16.9 us beside eight rows a warp), and more where
  // few units can be cut: in calls of up to 8192 rows and 64 pairs of a request and a KV head four rows a warp,
  // two for up to four requests or where a mean request has full units.  Graph replays with eight, four and two
  // over 2048 keys: 64 query heads and 8 KV heads of 64, 1 x 8 rows 29.0 us, 22.7, 19.1; 4 x 16 30.5, 27.7, 27.8; 8 x
  // 16 31.6, 30.2, 31.2; 64 x 1 61.5, 62.4, 65.3; 32 query heads and 4 KV heads of 128, 8 x 16 35.5, 32.6, 32.8; 64 x 1
  // 55.0, 55.3, 57.8; 16 heads of 64 to query and KV, 64 x 1 110, 109, 106 (8 CTAs with two).
  const int rows = static_cast<int>(
      std::min<long long>(static_cast<long long>(p.c.T) * (p.c.H / p.c.G), p.part_rows));
  const long long all = static_cast<long long>(p.c.T) * p.c.H, pairs = static_cast<long long>(p.c.B) * p.c.G;
  int per_warp = rows <= 32 ? 1 : rows <= 64 ? 2 : rows <= 128 ? 4 : 8;
  if (all <= 8192 && pairs <= 64)
    per_warp = std::min(per_warp, (p.c.B <= 4 && pairs <= 32) || all / pairs >= kUnitRows ? 2 : 4);
  const int join = (rows + 4 * per_warp - 1) / (4 * per_warp);
  return launch_chained(chunk_join_kernel<HD, kTree>, dim3(p.grid, join), dim3(128), 0, st, p) == cudaSuccess
             ? PE_OK
             : PE_ERR_CUDA;
}

}  // namespace

bool chunk_tc_takes(const pe_attn_plan* plan) {
  return plan->dtype == PE_DTYPE_BF16 && plan->block_size % 8 == 0;
}

size_t chunk_tc_workspace(const pe_attn_plan* plan, int max_rows) {
  const int rows = part_rows_of(max_rows, plan->n_heads / plan->n_kv_heads);
  return 256 + rec_bytes() + ml_bytes(rows) +
         al256(size_t{kMaxGrid} * 2 * rows * plan->head_dim * sizeof(float));
}

int launch_chunk_tc(const ChunkArgs& a, const TreeMask& mask, char* ws, cudaStream_t st) {
  TcTreeArgs p = {};
  p.mask = mask;
  p.c = a;
  p.box = 8;
  const int tile = a.hd == 64 ? Shape<64>::kTile : Shape<128>::kTile;
  while (p.box < tile && a.bs % (2 * p.box) == 0) p.box *= 2;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return PE_ERR_CUDA;
  p.grid = sms < kMaxGrid ? sms : kMaxGrid;
  const int HG = a.H / a.G;
  p.hg_shift = -1;
  for (int i = 0; i < 8; ++i)
    if (HG == 1 << i) p.hg_shift = i;
  // The least piece: one token over 2048 keys of 8 KV heads takes 20.0 us with 3 tiles,
  // 19.6 with 4, 18.7 with 5, 19.1 with 6.  A unit costs a CTA the time of ten tiles
  // beside its own (Q, the first tile's way through the pipeline, its results): a prompt
  // of 8192 takes 642 us with 6, 604 with 8, 571 with 10, 568 with 12; 64 x 8 rows 108 to
  // 109 us up to 10, 111 above.
  p.umin = 5;
  p.overhead = 10;
  p.part_rows = part_rows_of(a.T, HG);
  p.rec = reinterpret_cast<Rec*>(ws + 256);
  p.part_ml = reinterpret_cast<float*>(ws + 256 + rec_bytes());
  p.part_o = reinterpret_cast<float*>(ws + 256 + rec_bytes() + ml_bytes(p.part_rows));
  CUtensorMap km, vm;
  const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * a.G * a.bs;
  auto* encode = a.hd == 64 ? encode_tmap_bf16 : encode_tmap_bf16_rows128;
  if (!encode(&km, a.k_cache, rows, a.hd, p.box) || !encode(&vm, a.v_cache, rows, a.hd, p.box))
    return PE_ERR_CUDA;
  if (mask.bits) return a.hd == 64 ? launch<64, true>(p, km, vm, st) : launch<128, true>(p, km, vm, st);
  return a.hd == 64 ? launch<64, false>(p, km, vm, st) : launch<128, false>(p, km, vm, st);
}

}  // namespace pe
