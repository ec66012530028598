// The pages of a cache: copied (pe_cache_copy), given to rows of the block table
// (pe_pages_reserve), shared between them (pe_pages_fork), given back (pe_pages_free), and the
// accepted nodes of a tree moved behind their context (pe_cache_compact).
//
// The caches are [n_layers][num_blocks][G][bs][hd]: a page of one layer is one run of G bs hd
// elements, the vector of one position and KV head one of hd.  Everything here moves bytes
// (16 at a time) or counts; nothing is computed.
//
// Free pages are those whose count is 0.  They are handed out in ascending order, to the
// calls' entries in order, so a call's outcome does not depend on how its CTAs run: one CTA
// per entry checks it and counts what it needs, the last of them to finish adds up and lists
// as many free pages, a second kernel fills in the rows and copies.  (64 forks of 8 prompts and the
// free before them, 14 MB in 16 layers: 15 us for the two calls, 14 of it host time; launched cold 6
// for the free, 9.3 for the check and the list, 9.4 for rows and copies.)
#include <algorithm>
#include <atomic>

#include "pe_common.cuh"
#include "pe_paged.h"

namespace pe {
namespace {

constexpr int kThreads = 256;
constexpr int kScanThreads = 512;  // of the kernel that checks and lists
constexpr int kMaxRow = 1 << 22;   // entries of a row of the table: kScanThreads rows' have an int's sum
constexpr int kBatch = 8;          // 16-byte loads in flight per thread
// The counter of finished CTAs: a place of its own among a workspace's first 256 bytes, where no other
// call writes anything but zeros (0: the status word, 128: pe_sample's list length), so that one
// workspace can serve several calls in turn.
constexpr int kDone = 192;

struct CacheArgs {
  int layers, num_blocks, G, bs;
  int cpv;       // 16-byte chunks of a vector of hd elements
  uint4* kc;
  uint4* vc;
  uint32_t* status;
};

// Untiled bulk copies back to global memory.
PE_DEV void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\tcp.async.bulk.commit_group;" ::"l"(dst),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
template <int N>
PE_DEV void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
PE_DEV void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// chunk 0 of position `off` of block blk, head g, layer l
PE_DEV int64_t chunk_at(const CacheArgs& c, int l, int64_t blk, int g, int off) {
  return (((static_cast<int64_t>(l) * c.num_blocks + blk) * c.G + g) * c.bs + off) * c.cpv;
}

// ------------------------------------------------------------------ copy

// Pieces of pages go through a ring in shared memory by bulk copies, by one thread of a CTA per
// SM: HBM is what bounds it (1001 pages of 16 layers, 1.05 GB read and written: 161 us, 6.5 TB/s;
// a plain copy of as many bytes in one piece 155).  64 KB of loads in flight an SM and as much
// of stores do: 4 slots or 6 of 8 KB take 192, 12 slots 164 to 167.  By threads, with two 16-byte
// loads each in many CTAs, it took 173, with more loads or fewer CTAs 178 to 234.
constexpr int kPiece = 16384;  // bytes
constexpr int kSlots = 8;
constexpr int kStores = 4;     // stores that may still read their slots

struct Piece {
  const char* from;
  char* to;
  uint32_t bytes;  // 0: nothing to copy
};

__global__ void __launch_bounds__(32) page_copy_kernel(const CacheArgs c, int n, const int32_t* src,
                                                       const int32_t* dst, int64_t pieces, int per_page) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t full[kSlots];
  pdl_trigger();
  if (threadIdx.x != 0) return;
  for (int i = 0; i < kSlots; ++i) mbar_init(&full[i], 1);
  fence_barrier_init();
  fence_proxy_async();
  pdl_wait();
  const int64_t page = static_cast<int64_t>(c.G) * c.bs * c.cpv * 16;  // bytes of a page
  // the pages of one layer one after another
  auto piece = [&](int64_t k) {
    const int64_t it = k / per_page, lk = it / n;
    const int i = static_cast<int>(it - lk * n);
    const int64_t at = (k - it * per_page) * kPiece;
    const int s = src[i], d = dst[i];
    Piece p{nullptr, nullptr, 0u};
    if (s < 0 || s >= c.num_blocks || d < 0 || d >= c.num_blocks) {
      set_status(c.status, PE_ST_BLOCK_RANGE);
    } else if (s != d) {
      char* base = reinterpret_cast<char*>(lk & 1 ? c.vc : c.kc) + (lk >> 1) * c.num_blocks * page + at;
      p.from = base + s * page;
      p.to = base + d * page;
      p.bytes = static_cast<uint32_t>(page - at < kPiece ? page - at : kPiece);
    }
    return p;
  };
  // the places of the loads in flight
  char* to[kSlots];
  uint32_t bytes[kSlots];
  int64_t next = blockIdx.x;
  uint32_t loads = 0, stores = 0;
  int never = 0;
  auto load = [&]() {
    for (; next < pieces; next += gridDim.x) {
      const Piece p = piece(next);
      if (p.bytes == 0) continue;
      const int slot = loads % kSlots;
      to[slot] = p.to;
      bytes[slot] = p.bytes;
      mbar_arrive_expect_tx(&full[slot], p.bytes);
      bulk_load(ring + slot * kPiece, p.from, p.bytes, &full[slot]);
      ++loads;
      next += gridDim.x;
      return;
    }
  };
  for (int i = 0; i < kSlots - kStores; ++i) load();
  while (stores < loads) {
    const int slot = stores % kSlots;
    if (!mbar_wait(&full[slot], stores / kSlots & 1, &never)) {
      set_status(c.status, PE_ST_TIMEOUT);
      break;
    }
    bulk_store(to[slot], ring + slot * kPiece, bytes[slot]);
    ++stores;
    // the slot of the store kStores ago is free
    bulk_wait_read<kStores>();
    load();
  }
  for (uint32_t i = stores; i < loads; ++i) mbar_wait(&full[i % kSlots], i / kSlots & 1, &never);
  bulk_wait_all();
}

// ------------------------------------------------------------------ compact

struct CompactArgs {
  CacheArgs c;
  int B, T, max_blocks;
  const int32_t* qsl;
  const int32_t* seq_len;
  const int32_t* accepted;
  const int32_t* path;
  const int32_t* block_table;
};

// Row d of a request's path goes from node path[d] to node d.  The path ascends, so
// d <= path[d], and a thread that moves its 16 bytes of each row in order (kBatch loads, then
// their stores) reads every node before it is written over: node e is written by row e, at or
// after the row that comes from it.  (64 requests, 14 MB read and written in 16 layers: 7 us a
// call, which is its host time; launched cold the kernel takes 9, of which the bytes are 2: a chain
// of offsets, path and block table comes before the first of them.)
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactArgs a) {
  constexpr int kRows = 256;  // of the path at a time
  __shared__ int64_t from_sh[kRows], to_sh[kRows];
  __shared__ int bad_sh;
  pdl_trigger();
  pdl_wait();
  const CacheArgs& c = a.c;
  const int r = blockIdx.y, tid = threadIdx.x;
  const RowRange x = request_rows(a.qsl, r, a.T);
  const int n = x.q1 - x.q0, want = a.accepted[r], acc = min(max(want, 0), max(n - 1, 0));
  uint32_t st = x.bad ? PE_ST_ROWS_RANGE : 0u;
  if (want != acc) st |= PE_ST_ACCEPTED_RANGE;
  if (tid == 0) bad_sh = 0;
  __syncthreads();
  for (int d = 1 + tid; d <= acc; d += kThreads) {
    const int p = a.path[x.q0 + d];
    if (p >= n || p <= (d == 1 ? 0 : a.path[x.q0 + d - 1])) bad_sh = 1;
  }
  __syncthreads();
  if (bad_sh) st |= PE_ST_TREE;
  const int moved = bad_sh ? 0 : acc;
  const int64_t ctx = static_cast<int64_t>(a.seq_len[r]) - n;
  // this thread's 16 bytes: of layer, keys or values, head
  const int64_t units = static_cast<int64_t>(c.layers) * 2 * c.G * c.cpv;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kThreads + tid;
  const int ch = static_cast<int>(unit % c.cpv), g = static_cast<int>(unit / c.cpv % c.G);
  const int64_t lk = unit / c.cpv / c.G;
  uint4* base = (lk & 1 ? c.vc : c.kc) + chunk_at(c, static_cast<int>(lk >> 1), 0, g, 0) + ch;
  // chunks from there to a position of the request, -1: it has no valid page
  auto place = [&](int64_t t) {
    const int64_t b = t / c.bs;
    const int blk = t < 0 || b >= a.max_blocks ? -1 : a.block_table[static_cast<int64_t>(r) * a.max_blocks + b];
    if (blk < 0 || blk >= c.num_blocks) {
      st |= PE_ST_BLOCK_RANGE;
      return int64_t{-1};
    }
    return chunk_at(c, 0, blk, 0, static_cast<int>(t % c.bs));
  };
  for (int d0 = 1; d0 <= moved; d0 += kRows) {
    const int rows = min(kRows, moved - d0 + 1);
    if (tid < rows) {
      const int p = a.path[x.q0 + d0 + tid];
      int64_t f = -1, t = -1;
      if (p != d0 + tid) {
        f = place(ctx + p);
        t = place(ctx + d0 + tid);
      }
      from_sh[tid] = t < 0 ? -1 : f;
      to_sh[tid] = t;
    }
    __syncthreads();
    if (unit < units) {
      for (int d = 0; d < rows; d += kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e)
          if (d + e < rows && from_sh[d + e] >= 0) v[e] = base[from_sh[d + e]];
#pragma unroll
        for (int e = 0; e < kBatch; ++e)
          if (d + e < rows && from_sh[d + e] >= 0) base[to_sh[d + e]] = v[e];
      }
    }
    __syncthreads();
  }
  if (st && blockIdx.x == 0) set_status(c.status, st);
}

// ------------------------------------------------------------------ reserve, fork, free

struct PoolArgs {
  int n, rows, max_blocks, num_blocks, bs;
  const int32_t* row;     // reserve, free: the table's rows; fork: the children
  const int32_t* parent;  // fork
  const int32_t* length;
  int32_t* table;
  int32_t* refs;
  uint32_t* status;
  uint32_t* done;   // CTAs of the checking kernel that finished; 0 between calls (the last CTA leaves it
                    // so, and the second kernel, whatever stood there before)
  int32_t* need;    // [n] pages that entry i needs, -1: it is refused
  int32_t* start;   // [n] its first one in list
  int32_t* list;    // [num_blocks] free pages
};

// Sum over the CTA (kScanThreads) before this thread, and of all.
PE_DEV int scan_before(int v, int* warps, int& all) {
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
  for (int w = 0; w < kScanThreads / 32; ++w) {
    if (w < warp) before += warps[w];
    all += warps[w];
  }
  return before;
}

// By the last CTA: each entry's place in the list of free pages, and the list.  Entries are
// served in order; the first whose pages are not there, and all later ones that need some, are
// refused.
PE_DEV void hand_out(const PoolArgs& a, int* warps) {
  const int tid = threadIdx.x;
  __shared__ int total_sh;
  int64_t total = 0;  // pages that the entries so far need
  for (int i0 = 0; i0 < a.n; i0 += kScanThreads) {
    const int i = i0 + tid;
    const int need = i < a.n ? max(__ldcg(a.need + i), 0) : 0;
    int all;
    const int64_t at = total + scan_before(need, warps, all);
    if (i < a.n) a.start[i] = at > a.num_blocks ? a.num_blocks : static_cast<int>(at);
    total += all;
  }
  // free pages, until there are as many (at most num_blocks) or no page is left
  const int most = static_cast<int>(total < a.num_blocks ? total : static_cast<int64_t>(a.num_blocks));
  int found = 0;
  for (int64_t b0 = 0; b0 < a.num_blocks && found < most; b0 += 4 * kScanThreads) {
    const int64_t b = b0 + 4 * tid;
    unsigned free4 = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (b + e < a.num_blocks && __ldcg(a.refs + b + e) == 0) free4 |= 1u << e;
    int all;
    int at = found + scan_before(__popc(free4), warps, all);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (free4 >> e & 1u) {
        if (at < most) a.list[at] = static_cast<int>(b + e);
        ++at;
      }
    found += all;
  }
  if (tid == 0) total_sh = min(found, most);
  __syncthreads();
  const int there = total_sh;
  bool out = false;
  for (int i = tid; i < a.n; i += kScanThreads) {
    const int need = __ldcg(a.need + i);
    if (need > 0 && a.start[i] + static_cast<int64_t>(need) > there) {
      a.need[i] = -1;
      out = true;
    }
  }
  if (out) set_status(a.status, PE_ST_PAGES);
}

// Whether this is the last CTA; the others' results are then visible.
PE_DEV bool last_cta(const PoolArgs& a) {
  __shared__ bool last_sh;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last_sh = atomicAdd(a.done, 1u) == static_cast<uint32_t>(a.n) - 1u;
    if (last_sh) *a.done = 0u;
    __threadfence();
  }
  __syncthreads();
  return last_sh;
}

// The k-th free page; -1 where there is none (in a workspace that was not zeroed anything may stand).
PE_DEV int listed(const PoolArgs& a, int k) {
  const int page = k >= 0 && k < a.num_blocks ? a.list[k] : -1;
  return page < a.num_blocks ? page : -1;
}

// The entries of a row of the table that a length needs, -1: it does not fit in a row.
PE_DEV int entries_of(const PoolArgs& a, int len) {
  const int e = len < 0 ? -1 : len / a.bs + (len % a.bs != 0);
  return e > a.max_blocks ? -1 : e;
}

__global__ void __launch_bounds__(kScanThreads) reserve_check_kernel(const PoolArgs a) {
  __shared__ int warps[kScanThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.x, tid = threadIdx.x;
  const int row = a.row[i], e = entries_of(a, a.length[i]);
  bool bad = row < 0 || row >= a.rows || e < 0;
  for (int j = tid; j < a.n; j += kScanThreads) bad |= j != i && a.row[j] == row;  // the same row twice
  bad = __syncthreads_or(bad);
  int missing = 0;
  if (!bad)
    for (int b = tid; b < e; b += kScanThreads) missing += a.table[static_cast<int64_t>(row) * a.max_blocks + b] < 0;
  int all;
  scan_before(missing, warps, all);
  if (tid == 0) {
    a.need[i] = bad ? -1 : all;
    if (bad) set_status(a.status, PE_ST_PAGES);
  }
  if (last_cta(a)) hand_out(a, warps);
}

__global__ void __launch_bounds__(kScanThreads) reserve_fill_kernel(const PoolArgs a) {
  __shared__ int warps[kScanThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.x, tid = threadIdx.x;
  if (i == 0 && tid == 0) *a.done = 0u;
  if (a.need[i] <= 0) return;
  const int e = entries_of(a, a.length[i]);
  int32_t* row = a.table + static_cast<int64_t>(a.row[i]) * a.max_blocks;
  int at = a.start[i];
  for (int b0 = 0; b0 < e; b0 += kScanThreads) {
    const int b = b0 + tid;
    const bool missing = b < e && row[b] < 0;
    int all;
    const int k = at + scan_before(missing, warps, all);
    if (missing) {
      const int page = listed(a, k);
      if (page >= 0) {
        row[b] = page;
        a.refs[page] = 1;
      }
    }
    at += all;
  }
}

// Fork i: an empty child row, no other entry's child or parent; a parent row with a page, in
// use, for every entry that the length needs.
__global__ void __launch_bounds__(kScanThreads) fork_check_kernel(const PoolArgs a) {
  __shared__ int warps[kScanThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.x, tid = threadIdx.x;
  const int child = a.row[i], parent = a.parent[i], len = a.length[i], e = entries_of(a, len);
  bool bad = child < 0 || child >= a.rows || parent < 0 || parent >= a.rows || e < 0;
  for (int j = tid; j < a.n; j += kScanThreads) bad |= a.parent[j] == child || (j != i && a.row[j] == child);
  bad = __syncthreads_or(bad);
  if (!bad) {
    const int32_t* to = a.table + static_cast<int64_t>(child) * a.max_blocks;
    const int32_t* from = a.table + static_cast<int64_t>(parent) * a.max_blocks;
    for (int b = tid; b < a.max_blocks; b += kScanThreads) {
      bad |= to[b] >= 0;
      if (b < e) {
        const int page = from[b];
        bad |= page < 0 || page >= a.num_blocks || __ldcg(a.refs + min(max(page, 0), max(a.num_blocks - 1, 0))) <= 0;
      }
    }
    bad = __syncthreads_or(bad);
  }
  if (tid == 0) {
    a.need[i] = bad ? -1 : len % a.bs != 0;
    if (bad) set_status(a.status, PE_ST_PAGES);
  }
  if (last_cta(a)) hand_out(a, warps);
}

// The child's row (first CTA of a fork), and the positions of its last page.
__global__ void __launch_bounds__(kThreads) fork_apply_kernel(const PoolArgs a, const CacheArgs c) {
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.y, tid = threadIdx.x;
  if (i == 0 && blockIdx.x == 0 && tid == 0) *a.done = 0u;
  const int need = a.need[i];
  if (need < 0) return;
  const int len = a.length[i], full = len / a.bs, part = len % a.bs;
  int32_t* to = a.table + static_cast<int64_t>(a.row[i]) * a.max_blocks;
  const int32_t* from = a.table + static_cast<int64_t>(a.parent[i]) * a.max_blocks;
  const int page = need ? listed(a, a.start[i]) : -1;
  if (need && page < 0) return;
  if (blockIdx.x == 0) {
    for (int b = tid; b < full; b += kThreads) {
      to[b] = from[b];
      atomicAdd(a.refs + from[b], 1);
    }
    if (tid == 0 && need) {
      to[full] = page;
      a.refs[page] = 1;
    }
  }
  if (!need) return;
  const int src = from[full];
  // runs of `part` positions, one for each layer, keys or values, head
  const int run = part * c.cpv;
  const int64_t chunks = static_cast<int64_t>(c.layers) * 2 * c.G * run;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t j = static_cast<int64_t>(blockIdx.x) * kThreads + tid; j < chunks; j += 4 * step) {
    uint4 v[4];
    uint4* d[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int64_t k = j + x * step;
      if (k >= chunks) continue;
      const int64_t u = k / run, lk = u / c.G;
      const int g = static_cast<int>(u % c.G), l = static_cast<int>(lk >> 1);
      uint4* base = (lk & 1 ? c.vc : c.kc) + k % run;
      v[x] = base[chunk_at(c, l, src, g, 0)];
      d[x] = base + chunk_at(c, l, page, g, 0);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (j + x * step < chunks) *d[x] = v[x];
  }
}

__global__ void __launch_bounds__(kThreads) free_kernel(const PoolArgs a) {
  pdl_trigger();
  pdl_wait();
  const int row = a.row[blockIdx.x];
  if (row < 0 || row >= a.rows) {
    if (threadIdx.x == 0) set_status(a.status, PE_ST_PAGES);
    return;
  }
  // (an exchange: a row that is named twice gives its pages back once)
  for (int b = threadIdx.x; b < a.max_blocks; b += kThreads) {
    int32_t* at = a.table + static_cast<int64_t>(row) * a.max_blocks + b;
    if (__ldcg(at) == -1) continue;
    const int page = atomicExch(at, -1);
    if (page < 0) continue;  // (there was none)
    if (page >= a.num_blocks) {
      set_status(a.status, PE_ST_BLOCK_RANGE);
    } else if (atomicSub(a.refs + page, 1) <= 0) {
      atomicAdd(a.refs + page, 1);  // (it was free: its count stays)
      set_status(a.status, PE_ST_PAGES);
    }
  }
}

// ------------------------------------------------------------------ host

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
size_t al256(size_t x) { return (x + 255) / 256 * 256; }

int elem_size(const pe_attn_plan* p) { return p->dtype == PE_DTYPE_BF16 ? 2 : 4; }

int cache_args(CacheArgs& c, const pe_attn_plan* plan, int n_layers, int num_blocks, void* k_cache, void* v_cache,
               void* ws) {
  if (!k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return PE_ERR_ARG;
  c.layers = n_layers;
  c.num_blocks = num_blocks;
  c.G = plan->n_kv_heads;
  c.bs = plan->block_size;
  c.cpv = plan->head_dim * elem_size(plan) / 16;
  c.kc = static_cast<uint4*>(k_cache);
  c.vc = static_cast<uint4*>(v_cache);
  c.status = static_cast<uint32_t*>(ws);
  return PE_OK;
}

bool ws_ok(const void* ws, size_t have, size_t want) { return ws && aligned(ws, 256) && have >= want; }

// offsets in a pool workspace: status, counter, then need, start and list
int pool_args(PoolArgs& a, int n, const int32_t* row, int rows, const int32_t* length, int32_t* table, int max_blocks,
              int num_blocks, int block_size, int32_t* refs, void* ws) {
  for (const void* p : {static_cast<const void*>(row), static_cast<const void*>(length),
                        static_cast<const void*>(table), static_cast<const void*>(refs)})
    if (!p || !aligned(p, 4)) return PE_ERR_ARG;
  a.n = n;
  a.rows = rows;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.bs = block_size;
  a.row = row;
  a.length = length;
  a.table = table;
  a.refs = refs;
  char* w = static_cast<char*>(ws);
  a.status = reinterpret_cast<uint32_t*>(w);
  a.done = reinterpret_cast<uint32_t*>(w + kDone);
  w += 256;
  a.need = reinterpret_cast<int32_t*>(w);
  w += al256(n * sizeof(int32_t));
  a.start = reinterpret_cast<int32_t*>(w);
  w += al256(n * sizeof(int32_t));
  a.list = reinterpret_cast<int32_t*>(w);
  return PE_OK;
}

}  // namespace
}  // namespace pe

using namespace pe;

extern "C" int pe_cache_copy(const pe_attn_plan* plan, int n_layers, int n, const int32_t* src, const int32_t* dst,
                             int num_blocks, void* k_cache, void* v_cache, void* ws, size_t ws_bytes,
                             void* stream) {
  NvtxRange nvtx("pe_cache_copy");
  if (!plan_ok(plan) || n_layers < 1 || n < 0 || num_blocks < 0 || !ws_ok(ws, ws_bytes, 256)) return PE_ERR_ARG;
  if (n == 0) return PE_OK;
  CacheArgs c = {};
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4) ||
      cache_args(c, plan, n_layers, num_blocks, k_cache, v_cache, ws) != PE_OK)
    return PE_ERR_ARG;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return PE_ERR_CUDA;
  // the function's shared-memory limit, once per device (a bit each; past 63 every time)
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PE_ERR_CUDA;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (!(set.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(page_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSlots * kPiece) !=
        cudaSuccess)
      return PE_ERR_CUDA;
    set.fetch_or(bit, std::memory_order_release);
  }
  const int64_t page = static_cast<int64_t>(c.G) * c.bs * c.cpv * 16;
  const int64_t per_page = (page + kPiece - 1) / kPiece, pieces = per_page * n * n_layers * 2;
  if (per_page > 0x7fffffff) return PE_ERR_UNSUPPORTED;
  const int grid = static_cast<int>(std::min<int64_t>(pieces, sms));
  return launch_chained(page_copy_kernel, dim3(grid), dim3(32), kSlots * kPiece, static_cast<cudaStream_t>(stream), c, n,
                        src, dst, pieces, static_cast<int>(per_page)) == cudaSuccess
             ? PE_OK
             : PE_ERR_CUDA;
}

extern "C" int pe_cache_compact(const pe_attn_plan* plan, int n_layers, int B, int T, const int32_t* qsl,
                                const int32_t* seq_len, const int32_t* accepted, const int32_t* path,
                                const int32_t* block_table, int max_blocks, int num_blocks, void* k_cache,
                                void* v_cache, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx("pe_cache_compact");
  if (!plan_ok(plan) || n_layers < 1 || B < 0 || T < 0 || max_blocks < 1 || num_blocks < 0 ||
      !ws_ok(ws, ws_bytes, 256))
    return PE_ERR_ARG;
  if (B > 65535) return PE_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return PE_OK;
  CompactArgs a = {};
  for (const void* p : {static_cast<const void*>(qsl), static_cast<const void*>(seq_len),
                        static_cast<const void*>(accepted), static_cast<const void*>(path),
                        static_cast<const void*>(block_table)})
    if (!p || !aligned(p, 4)) return PE_ERR_ARG;
  if (cache_args(a.c, plan, n_layers, num_blocks, k_cache, v_cache, ws) != PE_OK) return PE_ERR_ARG;
  a.B = B;
  a.T = T;
  a.max_blocks = max_blocks;
  a.qsl = qsl;
  a.seq_len = seq_len;
  a.accepted = accepted;
  a.path = path;
  a.block_table = block_table;
  const int64_t units = static_cast<int64_t>(n_layers) * 2 * a.c.G * a.c.cpv;
  const int64_t grid = (units + kThreads - 1) / kThreads;
  if (grid > 0x7fffffff) return PE_ERR_UNSUPPORTED;
  return launch_chained(compact_kernel, dim3(static_cast<unsigned>(grid), B), dim3(kThreads), 0,
                        static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? PE_OK
             : PE_ERR_CUDA;
}

extern "C" size_t pe_pages_workspace_bytes(int max_entries, int num_blocks) {
  if (max_entries < 0 || num_blocks < 0) return 0;
  return 256 + 2 * al256(max_entries * sizeof(int32_t)) + al256(num_blocks * sizeof(int32_t));
}

extern "C" int pe_pages_reserve(int n, const int32_t* row, const int32_t* length, int32_t* block_table, int rows,
                                int max_blocks, int num_blocks, int block_size, int32_t* refs, void* ws,
                                size_t ws_bytes, void* stream) {
  NvtxRange nvtx("pe_pages_reserve");
  if (n < 0 || rows < 0 || max_blocks < 1 || num_blocks < 0 || block_size < 1 ||
      !ws_ok(ws, ws_bytes, pe_pages_workspace_bytes(n, num_blocks)))
    return PE_ERR_ARG;
  if (n > 65535 || max_blocks >= kMaxRow) return PE_ERR_UNSUPPORTED;
  if (n == 0) return PE_OK;
  PoolArgs a = {};
  if (pool_args(a, n, row, rows, length, block_table, max_blocks, num_blocks, block_size, refs, ws) != PE_OK)
    return PE_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (launch_chained(reserve_check_kernel, dim3(n), dim3(kScanThreads), 0, st, a) != cudaSuccess) return PE_ERR_CUDA;
  return launch_chained(reserve_fill_kernel, dim3(n), dim3(kScanThreads), 0, st, a) == cudaSuccess ? PE_OK
                                                                                                   : PE_ERR_CUDA;
}

extern "C" int pe_pages_fork(const pe_attn_plan* plan, int n_layers, int n, const int32_t* parent,
                             const int32_t* child, const int32_t* length, int32_t* block_table, int rows,
                             int max_blocks, int num_blocks, int32_t* refs, void* k_cache, void* v_cache, void* ws,
                             size_t ws_bytes, void* stream) {
  NvtxRange nvtx("pe_pages_fork");
  if (!plan_ok(plan) || n_layers < 1 || n < 0 || rows < 0 || max_blocks < 1 || num_blocks < 0 ||
      !ws_ok(ws, ws_bytes, pe_pages_workspace_bytes(n, num_blocks)))
    return PE_ERR_ARG;
  if (n > 65535 || max_blocks >= kMaxRow) return PE_ERR_UNSUPPORTED;
  if (n == 0) return PE_OK;
  PoolArgs a = {};
  CacheArgs c = {};
  if (!parent || !aligned(parent, 4) ||
      pool_args(a, n, child, rows, length, block_table, max_blocks, num_blocks, plan->block_size, refs, ws) != PE_OK ||
      cache_args(c, plan, n_layers, num_blocks, k_cache, v_cache, ws) != PE_OK)
    return PE_ERR_ARG;
  a.parent = parent;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (launch_chained(fork_check_kernel, dim3(n), dim3(kScanThreads), 0, st, a) != cudaSuccess) return PE_ERR_CUDA;
  // CTAs of a fork: one round of loads per thread at half a page
  const int64_t chunks = static_cast<int64_t>(n_layers) * c.G * c.bs * c.cpv;
  const int per = static_cast<int>(std::min<int64_t>(std::max<int64_t>(chunks / (4 * kThreads), 1), 1024));
  return launch_chained(fork_apply_kernel, dim3(per, n), dim3(kThreads), 0, st, a, c) == cudaSuccess ? PE_OK
                                                                                                     : PE_ERR_CUDA;
}

extern "C" int pe_pages_free(int n, const int32_t* row, int32_t* block_table, int rows, int max_blocks,
                             int num_blocks, int32_t* refs, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx("pe_pages_free");
  if (n < 0 || rows < 0 || max_blocks < 1 || num_blocks < 0 || !ws_ok(ws, ws_bytes, 256)) return PE_ERR_ARG;
  if (max_blocks >= kMaxRow) return PE_ERR_UNSUPPORTED;
  if (n == 0) return PE_OK;
  PoolArgs a = {};
  if (!row || !block_table || !refs || !aligned(row, 4) || !aligned(block_table, 4) || !aligned(refs, 4))
    return PE_ERR_ARG;
  a.n = n;
  a.rows = rows;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.row = row;
  a.table = block_table;
  a.refs = refs;
  a.status = static_cast<uint32_t*>(ws);
  return launch_chained(free_kernel, dim3(n), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? PE_OK
             : PE_ERR_CUDA;
}
