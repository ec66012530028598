// A tree of drafts: what attention needs of it (pe_tree_layout) and the walk along the
// target's tokens (pe_tree_accept).
//
// Node j of a request is its row j of the batch; parent[j] < j, -1 for a node right behind
// the context.  The line of j is j, parent[j], parent[parent[j]], ...; a node stands at
// position ctx + (length of its line - 1), ctx = seq_len - n, and its keys and values lie at
// cache position ctx + j (siblings share a position, not a slot).
//
// Both kernels are one CTA per request, bound by latency: the parents go to shared memory at
// once, a thread per node follows its line there, and the walk looks for the next child among
// 32 nodes a step.  Children lie behind their parent, so all steps together pass over the
// nodes once.  (Launched cold: 16 nodes of one request 6 us and 5, 256 requests of 1 to 255
// nodes 9 and 7.5.  The two calls take 13 us together in either case, 12 of it host time.)
#include "pe_common.cuh"
#include "pe_paged.h"

namespace pe {
namespace {

constexpr int kThreads = 128;
constexpr int kNodes = PE_TREE_MAX_NODES;

struct TreeArgs {
  int B, T;
  const int32_t* qsl;
  const int32_t* parent;
  uint32_t* status;
  // layout
  const int32_t* seq_len;
  const int32_t* block_table;
  int max_blocks, num_blocks, bs, words;
  uint32_t* mask;
  int64_t* pos;
  int64_t* slot;
  // accept
  const int32_t* tok;
  const int32_t* target;
  int32_t* accepted;
  int32_t* path;
  int32_t* bonus;
};

// A parent that is no earlier node counts as none.
PE_DEV int checked_parent(int p, int j, uint32_t& st) {
  if (p >= -1 && p < j) return p;
  st |= PE_ST_TREE;
  return -1;
}

__global__ void __launch_bounds__(kThreads) tree_layout_kernel(const TreeArgs a) {
  __shared__ int up[kNodes];
  pdl_trigger();
  pdl_wait();
  const int r = blockIdx.x, tid = threadIdx.x;
  const RowRange x = request_rows(a.qsl, r, a.T);
  const int n = x.q1 - x.q0, m = min(n, 32 * a.words);  // nodes that have bits
  uint32_t st = (x.bad ? PE_ST_ROWS_RANGE : 0u) | (n > m ? PE_ST_TREE : 0u);
  const int64_t ctx = static_cast<int64_t>(a.seq_len[r]) - n;
  for (int j = tid; j < m; j += kThreads) up[j] = checked_parent(a.parent[x.q0 + j], j, st);
  __syncthreads();
  for (int j = tid; j < n; j += kThreads) {
    const int64_t row = x.q0 + j;
    uint32_t* mask = a.mask + row * a.words;
    int depth = 0, w = a.words - 1;
    if (j < m) {
      uint32_t bits = 0;
      int node = j;
      while (true) {  // (each parent is an earlier node: at most j steps)
        for (; w > node >> 5; --w) {
          mask[w] = bits;
          bits = 0;
        }
        bits |= 1u << (node & 31);
        if (up[node] < 0) break;
        node = up[node];
        ++depth;
      }
      mask[w--] = bits;
    }
    for (; w >= 0; --w) mask[w] = 0;
    const int64_t t = ctx + j;
    int64_t slot = PE_PADDING_SLOT_ID;
    if (j < m) {
      const int64_t b = t / a.bs;
      const int blk = t < 0 || b >= a.max_blocks ? -1 : a.block_table[static_cast<int64_t>(r) * a.max_blocks + b];
      if (blk >= 0 && blk < a.num_blocks)
        slot = static_cast<int64_t>(blk) * a.bs + t % a.bs;
      else
        st |= PE_ST_BLOCK_RANGE;
    }
    if (a.pos) a.pos[row] = ctx + depth;
    if (a.slot) a.slot[row] = slot;
  }
  if (st) set_status(a.status, st);
}

__global__ void __launch_bounds__(kThreads) tree_accept_kernel(const TreeArgs a) {
  __shared__ int up[kNodes], tok[kNodes], target[kNodes], path[kNodes];
  __shared__ int len_sh;
  pdl_trigger();
  pdl_wait();
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const RowRange x = request_rows(a.qsl, r, a.T);
  const int n = x.q1 - x.q0, m = min(n, kNodes);
  uint32_t st = (x.bad ? PE_ST_ROWS_RANGE : 0u) | (n > m ? PE_ST_TREE : 0u);
  for (int j = tid; j < m; j += kThreads) {
    up[j] = checked_parent(a.parent[x.q0 + j], j, st);
    tok[j] = a.tok[x.q0 + j];
    target[j] = a.target[x.q0 + j];
  }
  __syncthreads();
  if (tid < 32 && m > 0) {
    int cur = 0, len = 0;
    if (lane == 0) path[0] = 0;
    while (true) {
      // the first child with the target's token (a negative one: there is no token)
      const int want = target[cur];
      int next = -1;
      for (int j0 = (cur + 1) & ~31; j0 < m && want >= 0; j0 += 32) {
        const int j = j0 + lane;
        const unsigned hit = __ballot_sync(0xffffffffu, j > cur && j < m && up[j] == cur && tok[j] == want);
        if (hit) {
          next = j0 + __ffs(hit) - 1;
          break;
        }
      }
      if (next < 0) break;
      cur = next;
      ++len;
      if (lane == 0) path[len] = cur;
    }
    if (lane == 0) {
      len_sh = len;
      a.accepted[r] = len;
      a.bonus[r] = target[cur];
    }
  } else if (tid == 0) {
    len_sh = -1;
    a.accepted[r] = 0;
    a.bonus[r] = -1;
  }
  __syncthreads();
  const int len = len_sh;
  for (int j = tid; j < n; j += kThreads) a.path[x.q0 + j] = j <= len ? path[j] : -1;
  if (st) set_status(a.status, st);
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int check_rows(int B, int T, const void* qsl, const void* parent, const void* ws, size_t ws_bytes) {
  if (B < 0 || T < 0 || (B == 0 && T > 0)) return PE_ERR_ARG;
  if (B > 65535) return PE_ERR_UNSUPPORTED;
  if (!ws || !aligned(ws, 256) || ws_bytes < 256) return PE_ERR_ARG;
  if (B > 0 && (!qsl || !aligned(qsl, 4) || (T > 0 && !parent) || !aligned(parent, 4))) return PE_ERR_ARG;
  return PE_OK;
}

}  // namespace
}  // namespace pe

using namespace pe;

extern "C" int pe_tree_layout(int B, int T, const int32_t* qsl, const int32_t* seq_len, const int32_t* parent,
                              const int32_t* block_table, int max_blocks, int num_blocks, int block_size,
                              uint32_t* mask, int words, int64_t* pos, int64_t* slot, void* ws, size_t ws_bytes,
                              void* stream) {
  NvtxRange nvtx("pe_tree_layout");
  const int rc = check_rows(B, T, qsl, parent, ws, ws_bytes);
  if (rc != PE_OK) return rc;
  if (words < 1 || words > PE_TREE_MAX_NODES / 32 || max_blocks < 1 || num_blocks < 0 || block_size < 1)
    return PE_ERR_ARG;
  if (B == 0 || T == 0) return PE_OK;
  if (!seq_len || !block_table || !mask || !aligned(seq_len, 4) || !aligned(block_table, 4) || !aligned(mask, 4) ||
      !aligned(pos, 8) || !aligned(slot, 8))
    return PE_ERR_ARG;
  TreeArgs a = {};
  a.B = B;
  a.T = T;
  a.qsl = qsl;
  a.parent = parent;
  a.status = static_cast<uint32_t*>(ws);
  a.seq_len = seq_len;
  a.block_table = block_table;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.bs = block_size;
  a.words = words;
  a.mask = mask;
  a.pos = pos;
  a.slot = slot;
  return launch_chained(tree_layout_kernel, dim3(B), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a) ==
                 cudaSuccess
             ? PE_OK
             : PE_ERR_CUDA;
}

extern "C" int pe_tree_accept(int B, int T, const int32_t* qsl, const int32_t* parent, const int32_t* tok,
                              const int32_t* target, int32_t* accepted, int32_t* path, int32_t* bonus, void* ws,
                              size_t ws_bytes, void* stream) {
  NvtxRange nvtx("pe_tree_accept");
  const int rc = check_rows(B, T, qsl, parent, ws, ws_bytes);
  if (rc != PE_OK) return rc;
  if (B == 0) return PE_OK;
  if (!accepted || !bonus || (T > 0 && (!tok || !target || !path))) return PE_ERR_ARG;
  for (const void* p : {static_cast<const void*>(tok), static_cast<const void*>(target),
                        static_cast<const void*>(accepted), static_cast<const void*>(path),
                        static_cast<const void*>(bonus)})
    if (!aligned(p, 4)) return PE_ERR_ARG;
  TreeArgs a = {};
  a.B = B;
  a.T = T;
  a.qsl = qsl;
  a.parent = parent;
  a.status = static_cast<uint32_t*>(ws);
  a.tok = tok;
  a.target = target;
  a.accepted = accepted;
  a.path = path;
  a.bonus = bonus;
  return launch_chained(tree_accept_kernel, dim3(B), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a) ==
                 cudaSuccess
             ? PE_OK
             : PE_ERR_CUDA;
}
