// sfa_blocks.cu -- the blocks that requests hold: forking a request's blocks, giving blocks back,
// moving held blocks to the front of the pool, and the copies of cache rows that go with them.
//
// The pool is the one the step plan hands out from: free_blocks[taken ..] are free.  shares[x]
// counts the requests that hold block x beyond the first, so a block fresh from the free list has 0
// and the plan need not know of it.
//   fork      a request's whole blocks are shared (shares + 1), its last, partial one is copied
//   free      a block named m times with s shares is free when m > s, else it has s - m
//   compact   the k-th lowest free block takes the place of the k-th highest held one, while lower
// Every output is a function of the inputs alone: counts come from commutative atomics, the order of
// freed blocks from the first place that names them, ranks from prefix sums.
//
// compact runs as one cluster whose CTAs split the table's entries and the pool's bitmaps and meet
// at cluster barriers: no workspace, one launch.  A cluster barrier orders global memory too, for the
// cluster's threads; what another CTA wrote there is read past L1 (a fence of the GPU's scope before each
// barrier cost 0.6 us a call).
// Bound: latency (a chain of launch, lengths, table, block counters and the barriers between them)
// up to some 10^5 table entries; kv_copy_blocks: HBM.  On the device: fork of 8 and of 512 rows 4 and 5 us;
// free of 8384 table entries 9 us, of 718000 (323000 freed) 19; compact of 512 blocks 8 us, of 10000 blocks
// and 10200 entries 17; copies of 2500 blocks of 74 KB in each of two layers 107 us, 6.9 TB/s.
#include <algorithm>
#include <climits>

#include <cooperative_groups.h>

#include "sfa_internal.h"

namespace cg = cooperative_groups;

namespace sfa {
namespace {

__device__ __forceinline__ int warp_inclusive_sum(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// exclusive sum of v over the block's threads, the total in `total`; part: blockDim / 32 words
__device__ __forceinline__ int block_exclusive_sum(int v, int* part, int& total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  const int in = warp_inclusive_sum(v, lane);
  __syncthreads();   // part may still be read
  if (lane == 31) part[warp] = in;
  __syncthreads();
  const int w = lane < warps ? part[lane] : 0;   // (at most 32 warps)
  const int before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
  total = __reduce_add_sync(0xffffffffu, w);
  return before + in - v;
}

// blocks that `tokens` positions take, at most `most`
__device__ __forceinline__ int blocks_for(int tokens, int block_size, int most) {
  const unsigned n = ((unsigned)max(tokens, 0) + (unsigned)(block_size - 1)) / (unsigned)block_size;   // (below 2^32)
  return (int)min(n, (unsigned)most);
}

// the last entry e of the non-decreasing a[0..n) with a[e] <= x (a[0] <= x)
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------------------- fork
struct ForkParams {
  int32_t* table;
  int rows, max_blocks;
  int32_t* lens;
  const int32_t *src, *dst;
  int n;
  int32_t* shares;
  int num_blocks;
  const int32_t* free_blocks;
  int num_free;
  const int32_t* taken;
  int block_size;
  int32_t *copies, *taken_out;
  int* status;
};

constexpr int kForkThreads = 256, kForkItems = kForkThreads / 32;

// the positions that item i's source holds; -1 where the item is padding or names no row
__device__ __forceinline__ int fork_len(const ForkParams& p, int i, bool& bad) {
  const int s = p.src[i], d = p.dst[i];
  if (s < 0 || d < 0) return -1;
  if (s >= p.rows || d >= p.rows || s == d) {
    bad = true;
    return -1;
  }
  return (int)min((long long)max(p.lens[s], 0), min((long long)p.max_blocks * p.block_size, (long long)INT_MAX));
}

// a warp an item; how many items before it take a block, every CTA counts for itself
__global__ void __launch_bounds__(kForkThreads) blocks_fork_kernel(const ForkParams p) {
  __shared__ int part[kForkThreads / 32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int i0 = blockIdx.x * kForkItems, i = i0 + warp;
  bool ignored = false, bad = false, bad_block = false, none = false;
  int before = 0;
  for (int j = threadIdx.x; j < min(i0 + kForkItems, p.n); j += kForkThreads) {
    const int len = fork_len(p, j, ignored);
    if (j < i0 && len > 0 && len % p.block_size != 0) ++before;
  }
  int total;
  (void)block_exclusive_sum(before, part, total);
  const long long head = max(*p.taken, 0);
  long long at = head + total;   // the free entry of this item, if it takes one
  for (int j = i0; j < i0 + kForkItems && j < p.n; ++j) {
    const int len = fork_len(p, j, ignored);
    if (j == i) break;
    if (len > 0 && len % p.block_size != 0) ++at;
  }
  if (i < p.n) {
    const int len = fork_len(p, i, bad);
    int c[3] = {-1, -1, -1};
    if (len >= 0) {
      const int s = p.src[i], d = p.dst[i];
      const int full = len / p.block_size, rows = len % p.block_size;
      const int32_t* from = p.table + (size_t)s * p.max_blocks;
      int32_t* to = p.table + (size_t)d * p.max_blocks;
      for (int j = lane; j < full; j += 32) {
        const int x = from[j];
        to[j] = x;
        if (x >= 0 && x < p.num_blocks) atomicAdd(p.shares + x, 1); else bad_block = true;
      }
      if (rows > 0) {
        const int x = from[full];
        const int fresh = at < p.num_free ? p.free_blocks[at] : -1;
        if (at >= p.num_free) none = true;
        const bool ok = x >= 0 && x < p.num_blocks && (fresh >= 0 && fresh < p.num_blocks);
        if (!ok && at < p.num_free) bad_block = true;
        if (lane == 0) to[full] = fresh;
        if (ok) {
          c[0] = x;
          c[1] = fresh;
          c[2] = rows;
        }
        ++at;
      }
      if (lane == 0) p.lens[d] = len;
    }
    if (lane < 3) p.copies[3 * (size_t)i + lane] = lane == 0 ? c[0] : lane == 1 ? c[1] : c[2];
    if (i == p.n - 1 && lane == 0) *p.taken_out = (int)min(at, max((long long)p.num_free, head));
  }
  if (bad || bad_block) report_status(p.status, kStatusBadBlock);
  if (none) report_status(p.status, kStatusNoBlocks);
}

// ---------------------------------------------------------------------------- free
struct FreeParams {
  const int32_t* table;
  const int32_t *held, *keep;
  int rows, max_blocks;
  int32_t* shares;
  int num_blocks;
  int32_t* free_blocks;
  int num_free;
  const int32_t* taken;
  int block_size;
  int32_t* taken_out;
  int* counts;                             // workspace [grid]: blocks that a CTA's entries put back
  int* status;
};

constexpr int kClusterThreads = 1024;
constexpr int kClusterCtas = 8;            // free: at most, of the form for small tables; compact: of the form for large ones
constexpr int kMarked = INT_MIN;           // shares of a freed block while the call runs: kMarked + e

// sums [rows + 1] of the entries per row, counted by `count(row)`; returns the total
template <class Count>
__device__ __forceinline__ int row_sums(int rows, int* sums, int* part, Count count) {
  const int per = (rows + blockDim.x - 1) / blockDim.x;
  const int r0 = min((int)threadIdx.x * per, rows), r1 = min(r0 + per, rows);
  int mine = 0;
  for (int r = r0; r < r1; ++r) mine += sums[r] = count(r);
  int total;
  int at = block_exclusive_sum(mine, part, total);
  for (int r = r0; r < r1; ++r) {
    const int n = sums[r];
    sums[r] = at;
    at += n;
  }
  if (threadIdx.x == 0) sums[rows] = total;
  __syncthreads();
  return total;
}

// The entries between the kept and the held positions, counted through the rows, are dealt to the
// CTAs in ranges, and four steps follow one another: every entry takes a share of its block; entries of
// blocks below zero leave the lowest entry's number there; a CTA counts the blocks that its
// entries put back; they go to their places.  kStep 0: one cluster does the four, barriers between
// them.  1 to 4: a launch each, since the next step needs all of the one before; a launch fetches
// the lengths and its first entries while the one before it ends.
// Bound: latency, three to four dependent accesses a step.  No warp meets more than kFreeHeld * 32
// entries at a time, which stay in registers from the table to the last step.  (A cluster for every table,
// its entries found and read again in each step: 323000 freed entries 295 us.)
constexpr int kFreeCtas = 152, kFreeHeld = 4, kFreeWarps = kClusterThreads / 32, kFreeRound = kFreeHeld * kClusterThreads;

template <int kStep>
__global__ void __launch_bounds__(kClusterThreads) blocks_free_kernel(const FreeParams p) {
  extern __shared__ int sums[];            // [rows + 1], then [rows]: where in the table a row's entries begin
  int* firsts = sums + p.rows + 1;
  __shared__ int part[kFreeWarps];
  __shared__ int puts_here;
  constexpr bool kAll = kStep == 0;
  auto meet = [] {
    if (gridDim.x > 1) cg::this_cluster().sync(); else __syncthreads();
  };
  const int rank = blockIdx.x, ctas = gridDim.x, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  if (!kAll) asm volatile("griddepcontrol.launch_dependents;");
  const int total = row_sums(p.rows, sums, part, [&](int r) {
    const int kept = blocks_for(p.keep[r], p.block_size, p.max_blocks);
    firsts[r] = r * p.max_blocks + kept;
    return max(0, blocks_for(p.held[r], p.block_size, p.max_blocks) - kept);
  });
  const int each = (total + ctas - 1) / ctas;
  const int e0 = (int)min((long long)rank * each, (long long)total), e1 = min(e0 + each, total);
  int x[kFreeHeld];                        // the blocks that the lane's entries name, -1 if none
  auto first = [&](int round) { return e0 + round * kFreeRound + warp * kFreeHeld * 32 + lane; };
  auto fetch = [&](int round) {
    const int e = first(round);
    int row[kFreeHeld] = {};
    for (int n = p.rows; n > 1;) {         // each row[u] begins the n rows in which entry u's is
      const int half = n >> 1;
#pragma unroll
      for (int u = 0; u < kFreeHeld; ++u)
        if (sums[row[u] + half] <= e + 32 * u) row[u] += half;
      n -= half;
    }
#pragma unroll
    for (int u = 0; u < kFreeHeld; ++u)
      x[u] = e + 32 * u < e1 ? p.table[firsts[row[u]] - sums[row[u]] + e + 32 * u] : -1;
#pragma unroll
    for (int u = 0; u < kFreeHeld; ++u)
      if (x[u] < 0 || x[u] >= p.num_blocks) x[u] = -1;
  };
  const int rounds = (e1 - e0 + kFreeRound - 1) / kFreeRound;
  fetch(0);
  if (!kAll) asm volatile("griddepcontrol.wait;" ::: "memory");
  bool bad = false;
  if (kAll || kStep == 1)
    for (int i = 0; i < rounds; ++i) {
      if (i > 0) fetch(i);
#pragma unroll
      for (int u = 0; u < kFreeHeld; ++u) {
        if (x[u] >= 0) atomicSub(p.shares + x[u], 1);
        else if (first(i) + 32 * u < e1) bad = true;
      }
    }
  if (kAll) meet();
  // below zero: free, and the first entry that names it puts it back
  if (kAll || kStep == 2)
    for (int i = 0; i < rounds; ++i) {
      if (i > 0) fetch(i);
      int v[kFreeHeld];
#pragma unroll
      for (int u = 0; u < kFreeHeld; ++u) v[u] = x[u] >= 0 ? __ldcg(p.shares + x[u]) : 0;
#pragma unroll
      for (int u = 0; u < kFreeHeld; ++u)
        if (v[u] < 0) {
          if (v[u] < -1 && v[u] > INT_MIN / 2) bad = true;   // given back more often than held
          atomicMin(p.shares + x[u], kMarked + first(i) + 32 * u);
        }
    }
  if (kAll) meet();
  auto puts = [&](int i, bool (&put)[kFreeHeld]) {           // how many of the lane's entries put a block back
    int n = 0;
#pragma unroll
    for (int u = 0; u < kFreeHeld; ++u) put[u] = x[u] >= 0 && __ldcg(p.shares + x[u]) == kMarked + first(i) + 32 * u;
#pragma unroll
    for (int u = 0; u < kFreeHeld; ++u) n += put[u];
    return n;
  };
  bool put[kFreeHeld];
  int all = 0, before = 0;
  if (kAll || kStep == 3) {
    int mine = 0;
    for (int i = 0; i < rounds; ++i) {
      if (i > 0) fetch(i);
      mine += puts(i, put);
    }
    (void)block_exclusive_sum(mine, part, all);
    if (threadIdx.x == 0) (kAll ? puts_here : p.counts[rank]) = all;
  }
  if (kAll) meet();
  if (kAll || kStep == 4) {
    int n = 0;
    if (threadIdx.x < ctas) n = kAll ? *cg::this_cluster().map_shared_rank(&puts_here, threadIdx.x) : __ldcg(p.counts + threadIdx.x);
    (void)block_exclusive_sum(threadIdx.x < rank ? n : 0, part, before);
    (void)block_exclusive_sum(n, part, all);
  }
  if (kAll || kStep == 4) {
    const int head = min(max(*p.taken, 0), p.num_free);
    int at = head - all + before;          // (-all may be below the list's begin)
    for (int i = 0; i < rounds; ++i) {
      if (i > 0) fetch(i);
      if (!kAll) (void)puts(i, put);
      unsigned votes[kFreeHeld];
      int mine = 0, n;
#pragma unroll
      for (int u = 0; u < kFreeHeld; ++u) mine += __popc(votes[u] = __ballot_sync(0xffffffffu, put[u]));
      int k = block_exclusive_sum(lane == 0 ? mine : 0, part, n);
      k = at + __shfl_sync(0xffffffffu, k, 0);
#pragma unroll
      for (int u = 0; u < kFreeHeld; ++u) {
        const int to = k + __popc(votes[u] & ((1u << lane) - 1));
        if (put[u]) {
          if (to >= 0) p.free_blocks[to] = x[u];
          p.shares[x[u]] = 0;
        }
        k += __popc(votes[u]);
      }
      at += n;
    }
    if (rank == 0 && threadIdx.x == 0) {
      if (all > head) report_status(p.status, kStatusNoBlocks);
      *p.taken_out = max(head - all, 0);
    }
  }
  if (bad) report_status(p.status, kStatusBadBlock);
  if (kAll) meet();                        // the others read puts_here
}

// ------------------------------------------------------------------------- compact
struct CompactParams {
  const int32_t* table;
  const int32_t* lens;
  int rows, max_blocks;
  const int32_t* shares;
  int num_blocks;
  const int32_t* free_blocks;
  int num_free;
  const int32_t* taken;
  int block_size, max_moves, words;        // words: bitmap words of a CTA
  int32_t *table_out, *shares_out, *free_out, *copies;
  int* status;
};

// shared memory of a CTA: words of held, free and filled (free blocks that take a held one's
// place), the held and free blocks of the CTA before each word, then the sums over the rows
template <int kCtas>
__global__ void __launch_bounds__(kClusterThreads) blocks_compact_kernel(const CompactParams p) {
  extern __shared__ unsigned smem_u[];
  unsigned *held = smem_u, *open = held + p.words, *filled = open + p.words;
  int *held_before = reinterpret_cast<int*>(filled + p.words), *open_before = held_before + p.words;
  int* sums = open_before + p.words;
  __shared__ int part[kClusterThreads / 32];
  __shared__ int n_held, n_open, n_now, n_moved;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = kCtas > 1 ? (int)cluster.block_rank() : 0;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int gid = rank * kClusterThreads + tid;
  constexpr int kAll = kCtas * kClusterThreads;
  auto meet = [&] {
    if (kCtas > 1) cluster.sync(); else __syncthreads();
  };
  auto remote = [&](auto* at, int c) { return kCtas > 1 ? cluster.map_shared_rank(at, c) : at; };
  const int head = min(max(*p.taken, 0), p.num_free);
  bool bad = false;

  for (int w = tid; w < p.words; w += kClusterThreads) held[w] = open[w] = 0;
  const int total = row_sums(p.rows, sums, part, [&](int r) { return blocks_for(p.lens[r], p.block_size, p.max_blocks); });
  meet();
  // what requests hold and what the list has
  for (int e = gid; e < total; e += kAll) {
    const int r = last_at_most(sums, p.rows, e);
    const int x = p.table[(size_t)r * p.max_blocks + (e - sums[r])];
    if (x < 0 || x >= p.num_blocks) {
      bad = true;
      continue;
    }
    const int w = x / 32;
    atomicOr(remote(held, w / p.words) + w % p.words, 1u << (x % 32));
  }
  for (int i = head + gid; i < p.num_free; i += kAll) {
    const int x = p.free_blocks[i];
    if (x < 0 || x >= p.num_blocks) {
      bad = true;
      continue;
    }
    const int w = x / 32;
    const unsigned was = atomicOr(remote(open, w / p.words) + w % p.words, 1u << (x % 32));
    if (was >> (x % 32) & 1) bad = true;   // listed twice
  }
  meet();
  // blocks before each word: a thread sums a run of words
  const int per = (p.words + kClusterThreads - 1) / kClusterThreads;
  const int w0 = min(tid * per, p.words), w1 = min(w0 + per, p.words);
  int nh = 0, no = 0;
  for (int w = w0; w < w1; ++w) {
    if (held[w] & open[w]) {               // held and listed as free: held
      bad = true;
      open[w] &= ~held[w];
    }
    nh += __popc(held[w]);
    no += __popc(open[w]);
  }
  int sum_h, sum_o;
  int ah = block_exclusive_sum(nh, part, sum_h);
  int ao = block_exclusive_sum(no, part, sum_o);
  for (int w = w0; w < w1; ++w) {
    held_before[w] = ah;
    open_before[w] = ao;
    ah += __popc(held[w]);
    ao += __popc(open[w]);
  }
  if (tid == 0) {
    n_held = sum_h;
    n_open = sum_o;
  }
  meet();
  int all_held = 0, base_open = 0;
  for (int c = 0; c < kCtas; ++c) {
    const int h = *remote(&n_held, c), o = *remote(&n_open, c);
    if (c < rank) base_open += o;
    all_held += h;
  }
  // held blocks before the words of CTA c
  auto base_held = [&](int c) {
    int n = 0;
    for (int d = 0; d < c; ++d) n += *remote(&n_held, d);
    return n;
  };
  const int my_base_held = base_held(rank);
  // pair up: a word a warp, a block a lane
  int moved = 0;
  for (int w = warp; w < p.words; w += kClusterThreads / 32) {
    const unsigned hw = held[w], ow = open[w], below = (1u << lane) - 1;
    const int x = (rank * p.words + w) * 32 + lane;
    const int hb = my_base_held + held_before[w] + __popc(hw & below);
    const int ob = base_open + open_before[w] + __popc(ow & below);
    bool fill = false, leave = false;
    if (ow >> lane & 1) {
      fill = ob < p.max_moves && ob < all_held - hb;
      if (fill) p.copies[3 * (size_t)ob + 1] = x;
    } else if (hw >> lane & 1) {
      const int k = all_held - hb - 1;     // held blocks above it
      leave = k < p.max_moves && k < ob;
      if (leave) {
        p.copies[3 * (size_t)k] = x;
        p.copies[3 * (size_t)k + 2] = p.block_size;
      }
    }
    const unsigned f = __ballot_sync(0xffffffffu, fill), l = __ballot_sync(0xffffffffu, leave);
    moved += __popc(l);
    if (lane == 0) {
      filled[w] = f;
      open[w] = (ow & ~f) | l;
    }
  }
  int sum_m;
  (void)block_exclusive_sum(lane == 0 ? moved : 0, part, sum_m);
  int nn = 0;
  for (int w = w0; w < w1; ++w) nn += __popc(open[w]);
  int sum_n;
  int an = block_exclusive_sum(nn, part, sum_n);
  for (int w = w0; w < w1; ++w) {
    open_before[w] = an;                   // from here on: of the new free blocks
    an += __popc(open[w]);
  }
  if (tid == 0) {
    n_now = sum_n;
    n_moved = sum_m;
  }
  meet();
  int base_now = 0, all_now = 0, moves = 0;
  for (int c = 0; c < kCtas; ++c) {
    const int n = *remote(&n_now, c);
    if (c < rank) base_now += n;
    all_now += n;
    moves += *remote(&n_moved, c);
  }
  // the pool
  for (int w = warp; w < p.words; w += kClusterThreads / 32) {
    const int x = (rank * p.words + w) * 32 + lane;
    const unsigned hw = held[w], ow = open[w];
    if (x >= p.num_blocks) continue;
    const bool leave = (hw & ow) >> lane & 1;
    if (ow >> lane & 1) {
      const long long at = (long long)head + base_now + open_before[w] + __popc(ow & ((1u << lane) - 1));
      if (at < p.num_free) p.free_out[at] = x;
    }
    if (leave) {
      const int k = all_held - (my_base_held + held_before[w] + __popc(hw & ((1u << lane) - 1))) - 1;
      p.shares_out[__ldcg(p.copies + 3 * (size_t)k + 1)] = p.shares[x];
      p.shares_out[x] = 0;
    } else if (!(filled[w] >> lane & 1)) {
      p.shares_out[x] = p.shares[x];
    }
  }
  for (int i = gid; i < p.num_free; i += kAll) {
    if (i < head) p.free_out[i] = p.free_blocks[i];
    else if (i >= head + all_now) p.free_out[i] = -1;
  }
  for (long long k = 3ll * moves + gid; k < 3ll * p.max_moves; k += kAll) p.copies[k] = -1;
  // the tables
  const long long entries = (long long)p.rows * p.max_blocks;
  for (long long e = gid; e < entries; e += kAll) {
    const int r = (int)(e / p.max_blocks), j = (int)(e % p.max_blocks);
    int x = p.table[e];
    if (j < sums[r + 1] - sums[r] && x >= 0 && x < p.num_blocks) {
      const int w = x / 32, c = w / p.words, i = w % p.words;
      const unsigned hw = remote(held, c)[i];
      if ((hw & remote(open, c)[i]) >> (x % 32) & 1) {
        const int k = all_held - (base_held(c) + remote(held_before, c)[i] + __popc(hw & ((1u << (x % 32)) - 1))) - 1;
        x = __ldcg(p.copies + 3 * (size_t)k + 1);
      }
    }
    p.table_out[e] = x;
  }
  if (bad) report_status(p.status, kStatusBadBlock);
  if (kCtas > 1) cluster.sync();           // bitmaps and counts are read by the others
}

// ---------------------------------------------------------------------------- copy
struct CopyParams {
  uint4* kv;
  float* scales;
  int layers, num_blocks, block_size, row_words, group;
  const int32_t* copies;
  int n;
  int chunks;                              // of kCopyWords words a block
  int turns;                               // CTAs that take a chunk's layers by turns
  int* status;
};

constexpr int kCopyThreads = 256, kCopyPer = 4, kCopyWords = kCopyThreads * kCopyPer;
// Where copies and chunks alone make this many CTAs (the GPU holds 1216), each takes all layers of its chunk, so
// that an unused entry costs one CTA a chunk, not one a layer: 4096 unused entries of 61 layers 744 us with one a
// layer, 13 so; 2000 used ones 2567 and 2625, 3000 of 4000 in 6 layers 103 and 101.  (With 32768: 28, 2601, 111.)
constexpr int kCopyCtas = 8192;

// a CTA a chunk of 16 KB of one copy, in every turns-th layer (kOne: in one layer; the loop costs 512 copies in 6
// layers 2 of 16 us)
template <bool kOne>
__global__ void __launch_bounds__(kCopyThreads) kv_copy_blocks_kernel(const CopyParams p) {
  const unsigned each = blockIdx.x / (unsigned)p.chunks, turn = each / (unsigned)p.n;
  const int chunk = (int)(blockIdx.x - each * (unsigned)p.chunks);
  const size_t item = each - turn * (unsigned)p.n;
  const int src = p.copies[3 * item], dst = p.copies[3 * item + 1];
  const int rows = min(max(p.copies[3 * item + 2], 0), p.block_size);
  if (src < 0) return;
  if (src >= p.num_blocks || dst < 0 || dst >= p.num_blocks) {
    if (threadIdx.x == 0) report_status(p.status, kStatusBadBlock);
    return;
  }
  const size_t block_words = (size_t)p.block_size * p.row_words;
  const long long end = (long long)rows * p.row_words, at = (long long)chunk * kCopyWords + threadIdx.x;
  int layer = (int)turn;
  do {
    const uint4* from = p.kv + ((size_t)layer * p.num_blocks + src) * block_words;
    uint4* to = p.kv + ((size_t)layer * p.num_blocks + dst) * block_words;
    uint4 x[kCopyPer];
#pragma unroll
    for (int u = 0; u < kCopyPer; ++u)
      if (at + u * kCopyThreads < end) x[u] = from[at + u * kCopyThreads];
#pragma unroll
    for (int u = 0; u < kCopyPer; ++u)
      if (at + u * kCopyThreads < end) to[at + u * kCopyThreads] = x[u];
    if (p.scales && chunk == 0) {
      const int per = p.block_size / p.group, n = (rows + p.group - 1) / p.group;
      for (int g = threadIdx.x; g < n; g += kCopyThreads)
        p.scales[((size_t)layer * p.num_blocks + dst) * per + g] = p.scales[((size_t)layer * p.num_blocks + src) * per + g];
    }
  } while (!kOne && (layer += p.turns) < p.layers);
}

constexpr int kUnasked = 40 * 1024;        // dynamic shared memory that a launch has beside the kernels' own
constexpr int kFreeMaxSmem = (2 * kPlanMaxRequests + 1) * 4;
constexpr int kCompactMaxSmem = (kMaxPoolBlocks / 32 / kClusterCtas) * 20 + (kPlanMaxRequests + 1) * 4;

// What a kernel may take is the kernel's, not the launch's: always the most that any call takes, so that a
// call on another host thread cannot lower it between this and the launch.
template <class Kernel>
cudaError_t allow_smem(Kernel kernel, int most) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

// after: begins while the launch before it on the stream ends (and waits for it itself)
template <class Kernel, class Params>
cudaError_t launch_ctas(Kernel kernel, int ctas, int cluster, size_t smem, const Params& p, cudaStream_t stream,
                        bool after = false) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kClusterThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_blocks_fork(int32_t* table, int rows, int max_blocks, int32_t* lens, const int32_t* src,
                               const int32_t* dst, int n, int32_t* shares, int num_blocks, const int32_t* free_blocks,
                               int num_free, const int32_t* taken, int block_size, int32_t* copies, int32_t* taken_out,
                               int* status, cudaStream_t stream) {
  if (n == 0) return cudaMemcpyAsync(taken_out, taken, 4, cudaMemcpyDeviceToDevice, stream);
  const ForkParams p{table, rows, max_blocks, lens, src, dst, n, shares, num_blocks, free_blocks,
                     num_free, taken, block_size, copies, taken_out, status};
  blocks_fork_kernel<<<(n + kForkItems - 1) / kForkItems, kForkThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

// CTAs: one for each round of the table's entries, up to a cluster (one launch); else one for each
// kClusterThreads entries, at most one for each SM.  2540 entries take 6.8 us by the cluster and 8.8 by
// the four launches, 8128 10.1 and 9.2, 31750 10.8 and 9.7 in a captured graph; called one by one, a
// cluster's call takes 16 us and four launches 25.
static int free_ctas(int rows, int max_blocks) {
  const long long entries = (long long)rows * max_blocks;
  if (entries <= kClusterCtas * kFreeRound) return std::max(1, (int)((entries + kFreeRound - 1) / kFreeRound));
  return (int)std::min<long long>((entries + kClusterThreads - 1) / kClusterThreads, kFreeCtas);
}

size_t blocks_free_workspace_bytes(int rows, int max_blocks) {
  const int ctas = free_ctas(rows, max_blocks);
  return ctas > kClusterCtas ? (size_t)ctas * 4 : 0;
}

cudaError_t launch_blocks_free(const int32_t* table, const int32_t* held, const int32_t* keep, int rows,
                               int max_blocks, int32_t* shares, int num_blocks, int32_t* free_blocks, int num_free,
                               const int32_t* taken, int block_size, int32_t* taken_out, void* workspace, int* status,
                               cudaStream_t stream) {
  const FreeParams p{table, held, keep, rows, max_blocks, shares, num_blocks, free_blocks, num_free, taken,
                     block_size, taken_out, static_cast<int*>(workspace), status};
  const size_t smem = (size_t)(2 * rows + 1) * 4;
  const int ctas = free_ctas(rows, max_blocks);
  const bool ask = smem > kUnasked;
  cudaError_t e = cudaSuccess;
  if (ctas <= kClusterCtas) {
    if (ask) e = allow_smem(blocks_free_kernel<0>, kFreeMaxSmem);
    return e != cudaSuccess ? e : launch_ctas(blocks_free_kernel<0>, ctas, ctas, smem, p, stream);
  }
  // for all four before the first, which already changes the shares
  if (ask)
    for (auto kernel : {blocks_free_kernel<1>, blocks_free_kernel<2>, blocks_free_kernel<3>, blocks_free_kernel<4>})
      if (e == cudaSuccess) e = allow_smem(kernel, kFreeMaxSmem);
  if (e == cudaSuccess) e = launch_ctas(blocks_free_kernel<1>, ctas, 1, smem, p, stream);
  if (e == cudaSuccess) e = launch_ctas(blocks_free_kernel<2>, ctas, 1, smem, p, stream, true);
  if (e == cudaSuccess) e = launch_ctas(blocks_free_kernel<3>, ctas, 1, smem, p, stream, true);
  if (e == cudaSuccess) e = launch_ctas(blocks_free_kernel<4>, ctas, 1, smem, p, stream, true);
  return e;
}

cudaError_t launch_blocks_compact(const int32_t* table, const int32_t* lens, int rows, int max_blocks,
                                  const int32_t* shares, int num_blocks, const int32_t* free_blocks, int num_free,
                                  const int32_t* taken, int block_size, int max_moves, int32_t* table_out,
                                  int32_t* shares_out, int32_t* free_out, int32_t* copies, int* status,
                                  cudaStream_t stream) {
  // by one CTA and by a cluster: 128 blocks 7.2 and 12.3 us, 4000 blocks and 3400 entries 13.9 and 15.5,
  // 10000 blocks and 10200 entries 26.7 and 17.4
  const bool small = (long long)rows * max_blocks <= 4 * kClusterThreads && num_blocks <= 8 * kClusterThreads;
  const int ctas = small ? 1 : kClusterCtas;
  const int all = (num_blocks + 31) / 32, words = (all + ctas - 1) / ctas;
  const CompactParams p{table, lens, rows, max_blocks, shares, num_blocks, free_blocks, num_free, taken, block_size,
                        max_moves, words, table_out, shares_out, free_out, copies, status};
  const size_t smem = (size_t)words * 20 + (size_t)(rows + 1) * 4;
  if (small) return launch_ctas(blocks_compact_kernel<1>, 1, 1, smem, p, stream);   // (at most 22 KB)
  if (smem > kUnasked) {
    const cudaError_t e = allow_smem(blocks_compact_kernel<kClusterCtas>, kCompactMaxSmem);
    if (e != cudaSuccess) return e;
  }
  return launch_ctas(blocks_compact_kernel<kClusterCtas>, kClusterCtas, kClusterCtas, smem, p, stream);
}

cudaError_t launch_kv_copy_blocks(void* kv, float* scales, int group, int row_bytes, int layers, int num_blocks,
                                  int block_size, const int32_t* copies, int n, int* status, cudaStream_t stream) {
  const int row_words = row_bytes / 16;
  const long long chunks = ((long long)block_size * row_words + kCopyWords - 1) / kCopyWords;
  if (n == 0 || layers == 0) return cudaSuccess;
  const long long most = std::min<long long>(layers, (kCopyCtas + chunks * n - 1) / (chunks * n));
  const long long each = (layers + most - 1) / most, turns = (layers + each - 1) / each;   // layers of a CTA
  const long long grid = chunks * n * turns;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  const CopyParams p{static_cast<uint4*>(kv), scales, layers, num_blocks, block_size, row_words, group, copies, n,
                     (int)chunks, (int)turns, status};
  (turns == layers ? kv_copy_blocks_kernel<true> : kv_copy_blocks_kernel<false>)<<<(unsigned)grid, kCopyThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace sfa
