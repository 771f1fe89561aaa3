// sfa_tree.cu -- a step that verifies a tree of drafted tokens, around its attention: the nodes'
// masks and positions from their parents, the accepted path, and the move of its cache rows to
// consecutive positions.
//
// Request b drafts n_b nodes, the tokens [token_start[b], token_start[b + 1]) of the step; node j's
// row lies at position cached_lens[b] + j of its sequence, whatever its depth.  parents[t] is a
// node's parent by its number within the request (smaller than its own), or -1.
//   plan    mask_i = mask_parent | bit i;  position_i = cached + depth_i
//   accept  from node 0 on: the first child whose token is its parent's target
//   commit  row of path[k] -> position cached + k
// Bound: latency.  A request's few hundred bytes of parents, tokens and targets go to shared memory
// in one round of loads, and the chains of parents and children are walked there.  Alone on the device,
// about 2 us of each being the launch: 64 requests of 4 to 8 nodes 4.0 us (plan), 3.7 (accept) and 5.8
// (commit); 256 of 30 to 61 nodes 4.9, 5.3 and 8.8 (the moved rows are 2 MB).
#include "sfa_internal.h"

namespace sfa {
namespace {

// the request's tokens, clipped to the step's
__device__ __forceinline__ void node_range(const int32_t* token_start, int b, int T, int& first, int& n) {
  first = min(max(token_start[b], 0), T);
  n = min(max(token_start[b + 1], first), T) - first;
}

struct TreePlanParams {
  const int32_t *parents, *token_start, *cached;
  int B, T, max_nodes, words;
  long long* mask;
  int32_t* positions;
  int* status;
};

constexpr int kPadTokens = 1024;   // tokens that a block of padding looks at

// block b < B: a thread for each node of request b; the blocks behind: tokens of no request
__global__ void tree_plan_kernel(const TreePlanParams p) {
  __shared__ int par[kTreeMaxNodes];
  if ((int)blockIdx.x >= p.B) {
    const int from = min(max(p.token_start[0], 0), p.T), to = min(max(p.token_start[p.B], 0), p.T);
    const int t0 = ((int)blockIdx.x - p.B) * kPadTokens;
    for (int t = t0 + threadIdx.x; t < min(t0 + kPadTokens, p.T); t += blockDim.x) {
      if (t >= from && t < to) continue;
      p.positions[t] = -1;
      for (int w = 0; w < p.words; ++w) p.mask[(size_t)t * p.words + w] = 0;
    }
    return;
  }
  int first, n;
  node_range(p.token_start, blockIdx.x, p.T, first, n);
  const int most = min(n, p.max_nodes);
  bool bad = n > p.max_nodes;
  const int cached = max(p.cached[blockIdx.x], 0);
  for (int i = threadIdx.x; i < most; i += blockDim.x) par[i] = p.parents[first + i];
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    unsigned long long m[kTreeMaxNodes / 64] = {};
    int depth = -1;
    if (i < most)
      for (int j = i; j >= 0; ++depth) {
#pragma unroll
        for (int w = 0; w < kTreeMaxNodes / 64; ++w)
          if (w == j / 64) m[w] |= 1ull << (j % 64);
        int up = par[j];
        if (up >= j || up < -1) {   // no tree: the node counts as a root
          bad = true;
          up = -1;
        }
        j = up;
      }
    p.positions[first + i] = depth < 0 ? -1 : cached + depth;
#pragma unroll
    for (int w = 0; w < kTreeMaxNodes / 64; ++w)
      if (w < p.words) p.mask[(size_t)(first + i) * p.words + w] = (long long)m[w];
  }
  if (bad) report_status(p.status, kStatusBadTree);
}

struct TreeAcceptParams {
  const int32_t *tokens, *targets, *parents, *token_start, *cached;
  int B, T, max_nodes;
  int32_t *path, *accepted, *next_tokens, *seq_lens;
  int* status;
};

constexpr int kAcceptWarps = 4;

// a warp a request
__global__ void __launch_bounds__(kAcceptWarps * 32) tree_accept_kernel(const TreeAcceptParams p) {
  __shared__ int tok_s[kAcceptWarps][kTreeMaxNodes], par_s[kAcceptWarps][kTreeMaxNodes],
      tgt_s[kAcceptWarps][kTreeMaxNodes];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int b = blockIdx.x * kAcceptWarps + warp;
  if (b >= p.B) return;
  int first, n;
  node_range(p.token_start, b, p.T, first, n);
  if (n > p.max_nodes) {
    if (lane == 0) report_status(p.status, kStatusBadTree);
    n = p.max_nodes;
  }
  const int cached = p.cached[b];
  for (int i = lane; i < n; i += 32) {
    tok_s[warp][i] = p.tokens[first + i];
    par_s[warp][i] = p.parents[first + i];
    tgt_s[warp][i] = p.targets[first + i];
  }
  __syncwarp();
  int32_t* path = p.path + (size_t)b * p.max_nodes;
  int count = 0, want = -1;
  // a child's number is above its parent's, so the walk ends
  for (int cur = n > 0 ? 0 : -1; cur >= 0;) {
    if (lane == 0) path[count] = cur;
    ++count;
    want = tgt_s[warp][cur];
    int next = -1;
    for (int j0 = cur + 1; j0 < n && next < 0; j0 += 32) {
      const int j = j0 + lane;
      const unsigned hit = __ballot_sync(0xffffffffu, j < n && par_s[warp][j] == cur && tok_s[warp][j] == want);
      if (hit) next = j0 + __ffs(hit) - 1;
    }
    cur = next;
  }
  for (int i = count + lane; i < p.max_nodes; i += 32) path[i] = -1;
  if (lane == 0) {
    p.accepted[b] = count;
    p.next_tokens[b] = want;
    p.seq_lens[b] = max(cached, 0) + count;
  }
}

struct CommitParams {
  uint4* kv;
  int layers, num_blocks, block_size;
  const int32_t* table;
  int max_blocks;
  const int32_t *cached, *path, *accepted;
  int B, max_nodes;
  int* status;
};

constexpr int kRowWords = kDQK * 2 / 16;   // 72 x 16 bytes a row: a thread each
constexpr int kRowsAtOnce = 4;             // rows a thread has in flight
constexpr int kCommitThreads = 4 * kRowWords;

// 72 threads a (layer, request); each moves its 16 bytes of every row, in the order of the path, four rows
// in flight.
// Rows only move down (path ascends, path[k] >= k), so a row is read before its place is taken.
__global__ void __launch_bounds__(kCommitThreads) kv_commit_kernel(const CommitParams p) {
  const long long item = (long long)blockIdx.x * 4 + threadIdx.x / kRowWords;
  const int word = threadIdx.x % kRowWords;
  if (item >= (long long)p.layers * p.B) return;
  const int b = (int)(item % p.B), layer = (int)(item / p.B);
  const int n = min(max(p.accepted[b], 0), p.max_nodes);
  const long long cached = max(p.cached[b], 0);
  const int32_t* path = p.path + (size_t)b * p.max_nodes;
  const int32_t* table = p.table + (size_t)b * p.max_blocks;
  bool bad_tree = false, bad_block = false;
  auto at = [&](long long pos) -> uint4* {
    const long long blk = pos / p.block_size;
    const int phys = blk < p.max_blocks ? table[blk] : -1;
    if (phys < 0 || phys >= p.num_blocks) {
      bad_block = true;
      return nullptr;
    }
    return p.kv + (((size_t)layer * p.num_blocks + phys) * p.block_size + pos % p.block_size) * kRowWords + word;
  };
  int last = -1;
  for (int k0 = 0; k0 < n && !bad_tree; k0 += kRowsAtOnce) {
    uint4 x[kRowsAtOnce];
    uint4* to[kRowsAtOnce];
#pragma unroll
    for (int u = 0; u < kRowsAtOnce; ++u) {
      const int k = k0 + u;
      to[u] = nullptr;
      if (k >= n || bad_tree) continue;
      const int from = path[k];
      if (from <= last || from >= kTreeMaxNodes) {
        bad_tree = true;
        continue;
      }
      last = from;
      if (from == k) continue;
      const uint4* src = at(cached + from);
      uint4* dst = at(cached + k);
      if (!src || !dst) continue;
      x[u] = *src;
      to[u] = dst;
    }
#pragma unroll
    for (int u = 0; u < kRowsAtOnce; ++u)
      if (to[u]) *to[u] = x[u];
  }
  if (word == 0 && bad_tree) report_status(p.status, kStatusBadTree);
  if (word == 0 && bad_block) report_status(p.status, kStatusBadBlock);
}

}  // namespace

cudaError_t launch_tree_plan(const int32_t* parents, const int32_t* token_start, const int32_t* cached, int B, int T,
                             int max_nodes, long long* mask, int32_t* positions, int* status, cudaStream_t stream) {
  const TreePlanParams p{parents, token_start, cached, B, T, max_nodes, (max_nodes + 63) / 64, mask, positions, status};
  if (T == 0) return cudaSuccess;
  const int threads = max_nodes <= 32 ? 32 : max_nodes <= 64 ? 64 : 128;
  tree_plan_kernel<<<B + (T + kPadTokens - 1) / kPadTokens, threads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_tree_accept(const int32_t* tokens, const int32_t* targets, const int32_t* parents,
                               const int32_t* token_start, const int32_t* cached, int B, int T, int max_nodes,
                               int32_t* path, int32_t* accepted, int32_t* next_tokens, int32_t* seq_lens, int* status,
                               cudaStream_t stream) {
  const TreeAcceptParams p{tokens, targets, parents, token_start, cached, B, T, max_nodes,
                           path, accepted, next_tokens, seq_lens, status};
  if (B == 0) return cudaSuccess;
  tree_accept_kernel<<<(B + kAcceptWarps - 1) / kAcceptWarps, kAcceptWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv_commit(void* kv, int layers, int num_blocks, int block_size, const int32_t* table,
                             int max_blocks, const int32_t* cached, const int32_t* path, const int32_t* accepted,
                             int B, int max_nodes, int* status, cudaStream_t stream) {
  const CommitParams p{static_cast<uint4*>(kv), layers, num_blocks, block_size, table, max_blocks, cached, path,
                       accepted, B, max_nodes, status};
  const long long items = (long long)layers * B;
  if (items == 0) return cudaSuccess;
  if ((items + 3) / 4 > 0x7fffffffLL) return cudaErrorInvalidValue;
  kv_commit_kernel<<<(unsigned)((items + 3) / 4), kCommitThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace sfa
