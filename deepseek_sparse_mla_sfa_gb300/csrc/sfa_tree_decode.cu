// sfa_tree_decode.cu -- tcgen05 / TMA path of the attention of drafted trees on sm_103a.
//
// All nodes of a request attend to the same cached rows, so a request's n_b nodes x h heads are the
// n_b * h rows of one dense attention whose keys and values are the request's c_b + n_b cache rows;
// only the columns of the nodes themselves carry a mask (a node's ancestors).
//
// Work.  A unit is 128 of those query rows (consecutive rows of q) of one request; its keys go by in
// tiles of 256 positions.  A pair of CTAs takes a tile with two-CTA MMAs (cta_group::2, M = 128): each
// CTA owns 64 query rows.  Per tile and CTA
//   S[64 x 256]  = q[64 x 576] K^T: the A operand is the CTA's q in shared memory, the B operand's 256
//                  keys lie half in either CTA, brought 64 columns at a time;
//   P = exp2(S - m), the CTA's own 64 rows, in shared memory, in one bf16 term, or in two (the value and
//                  what its rounding left) where the result is fp32;
//   O[64 x 512] += P V: either CTA holds the 256 value columns that its half of each N = 256 takes, of
//                  all 256 keys, brought 32 keys at a time; both halves of O take P from the collector.
// TMEM lanes 0-63 hold the CTA's 64 rows with the first half of an MMA's N, lanes 64-127 the same rows
// with the second half: O fills 256 columns, two score buffers the other 256.  One CTA's TMEM could not
// hold 128 rows of O and any scores; with 64 rows a CTA both fit, the softmax of a row stays in its CTA
// (four threads a row), and the pair reads each key once for 128 rows.  N = 256 in both products since
// an MMA of M = 128 takes 64 cycles for N = 256 and 66 for N = 128 (measured): tiles of 128 keys take
// 1.5 times as long a key.
//
// Order of the chunks (16 KB a CTA, a ring of 7, or of 5 beside two terms): K(0), then K(i+1), V(i) by
// turns, so QK^T of the next tile covers the softmax of this one.  The value columns of the CTA's own keys
// come twice (as keys and as values); the second time is from L2, which gives 180 GB/s an SM where the
// ring takes 80.
//
// Three launches: a block that lays out who works on what (the schedule, below), the pairs, and the joining
// of units that several pairs had parts of.
//
// Bound.  From 128 query rows a request on, the tensor cores: a tile of 256 keys is 4353 cycles of MMAs (6400
// with two terms), and takes 6200 to 6700 with its rows in L2 (keys awaited 700 to 1000, values 600, P 350;
// shared memory itself needs 5600 for the MMAs' and the loads' traffic).  16 requests x 16 nodes x 128 heads x
// 8192 positions, bf16 results: 418 us, 1399 TFLOP/s; 2 x 25 nodes x 64 heads x 131072 positions: 525 us,
// 1411.  With fewer rows the latency of memory: 64 x 2-8 nodes x 16 heads x 1000-16384 positions, fp32: 193 us
// where the bytes need 97; with all rows in L2 it takes 163, its products alone 101.  Short calls: latency, 18
// of the 27 us of 6 nodes x 4 heads x 200 positions in the pairs' launch (keys 7000 cycles, products and
// softmax 15000, the result 8000), the rest in the schedule and between the launches.
//
// Accuracy of fp32 results.  Scores and O are fp32 sums in the tensor core, which cuts each off towards zero: against
// 64 bits (2-norm) units of 250, 1000, 4000 and 16000 positions that one pair adds up are off by 1.1, 2.1, 4.3 and
// 7.4e-6, and 16000 positions cut over all pairs, whose parts are joined in registers, by 1.0e-6.
//
// Rows that nobody may see.  Positions behind the last node are brought as rows of zeros.  A cached row
// of NaN or infinities that only some nodes see would reach the others as 0 x NaN in P V: such a row
// shows as a score that is not finite in a masked place; the loading warps see a position that a node
// attends to and that has no block.  Both mark the request, a bit each, and the last kernel computes the
// nodes of every marked one on CUDA cores, once, which reads only what a node attends to.
//
// Warps (512 threads): 0-7 softmax, rescaling, output (the first thread brings q); 8 issues the MMAs (in
// the pair's first CTA) or fetches rows ahead (in the second); 9-15 bring keys and values, one a slot of the ring.  Every wait is bounded; one
// that gives up records SFA_ERR_DEVICE_TIMEOUT and both CTAs unwind.
#include <atomic>
#include <cuda.h>
#include <string.h>

#include "sfa_ptx.cuh"
#include "sfa_tree.cuh"

namespace sfa {
namespace {

using namespace ptx;

constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp = 9, kThreads = 16 * 32;
constexpr int kRows = 128, kHalf = 64;         // query rows of a unit, of a CTA
constexpr int kTile = 256;                     // positions of a tile
constexpr int kKChunks = 9, kVChunks = 8;      // of a tile
constexpr int kChunk = 16384;
constexpr int kUnitCost = 1;                   // of starting a unit, in tiles
// Cost a pair gets at least: a unit of one tile.  With 3, a pair could get the tiles of two units while
// others had none: 4 requests of 200 positions 39 us, with 2 28; 1 of 8000 positions x 16 heads 35 and 29.
constexpr int kMinSpan = 2;
constexpr int kMaxPairs = 128, kMaxSlots = 4 * kMaxPairs;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;      // log2 units: weights stay below 2^8

// shared memory (offsets from a 1024-byte aligned base): q, P (one bf16 term of the weights or two), the ring
constexpr int kQBlk = kHalf * 128;             // 64 rows x 64 columns
constexpr int kQBytes = 9 * kQBlk;
constexpr int kOffP = kQBytes;                 // P: four blocks of 64 rows x 64 keys a term
constexpr int kPBytes = 4 * kQBlk;
template <bool kTwo>
struct Ring {
  static constexpr int kSlots = kTwo ? 5 : 7;
  static constexpr int kOff = kOffP + (kTwo ? 2 : 1) * kPBytes;
  static_assert(kOff % 1024 == 0 && kOff + kSlots * kChunk == kOffP + kPBytes + 7 * kChunk, "the ring fills the rest");
};
constexpr int kOffMx = kOffP + kPBytes + 7 * kChunk;     // float [2][256]: row maxima, then sums
constexpr int kOffBar = kOffMx + 2048;
constexpr int kBarFull = 0, kBarEmpty = 7, kBarQFull = 14, kBarS = kBarQFull + 1, kBarP = kBarS + 2, kBarPv = kBarP + 1, kBarO = kBarPv + 1,
              kBarMx = kBarO + 1, kBarFin = kBarMx + 2, kBarNever = kBarFin + 1, kNumBars = kBarNever + 1;
constexpr int kOffMisc = kOffBar + 8 * kNumBars;         // TMEM address, abort
constexpr int kSmem = kOffMisc + 64 + 1024;
static_assert(kSmem <= 232448, "shared memory budget");
static_assert(kOffBar % 8 == 0, "alignment");

constexpr uint32_t kTmemCols = 512, kColO = 0, kColS = 256;
constexpr long long kDrainLimit = 1LL << 40;

// A part of a unit that one pair works through: its query rows and its tiles [k0, k1).
struct alignas(16) Piece {
  int row0, rows, k0, k1;
  int request, cached, n, first;       // the request, its cached positions, nodes and first token
  int slot;                            // of its partial result; -1: the piece is the whole unit
  int alone, pad[2];                   // the request's only unit
};
// a partial result: a unit's rows, and whether it has the unit's first tile
struct alignas(16) Partial {
  int row0, rows, request, begins;
};

struct Workspace {
  Piece* pieces;     // of pair k: [start[k], start[k + 1])
  int* start;        // [pairs + 1]
  int* partials;     // [1]: slots in use
  Partial* list;     // [slots]
  float* part;       // [slots][cap][512]
  float* lse;        // [slots][cap]
  unsigned* marks;   // [ceil(B / 32)]: a bit a request, which is to be computed on CUDA cores
  int cap, slots;    // rows of a slot, slots
  int most;          // pieces that there is room for
  __device__ __forceinline__ void mark(int request) const { atomicOr(marks + request / 32, 1u << (request % 32)); }
};

struct TreeTcParams {
  TreeParams p;
  Workspace ws;
  int pairs, num_rows, box;   // box: rows of a tiled load (0: rows one by one)
};

// ---------------------------------------------------------------- cta_group::2 forms
__device__ __forceinline__ void tmem_alloc2(uint32_t* dst, uint32_t n) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(n)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t a, uint32_t n) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(a), "r"(n) : "memory");
}
// Operand descriptors by their low words (address and leading offset); the high words (stride 1024,
// version 1, 128-byte swizzle) are the same for all.  From an elected lane of a converged warp, with
// uniform operands: 64-bit descriptors put together by one lane take it 80 to 140 cycles an MMA, more
// than the MMA.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (kSwizzle128 << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | (lbo >> 4) << 16; }
__device__ __forceinline__ void mma2(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
// two MMAs with one A, which the second takes from the collector
__device__ __forceinline__ void mma2_pair(uint32_t d0, uint32_t d1, uint32_t a, uint32_t b0, uint32_t b1, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db, dc;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 da, {%2, %7};\n\tmov.b64 db, {%3, %7};\n\tmov.b64 dc, {%4, %7};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16.collector::a::fill [%0], da, db, %5, p;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16.collector::a::lastuse [%1], da, dc, %5, p;\n\t}" ::"r"(d0),
      "r"(d1), "r"(a), "r"(b0), "r"(b1), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
// one lane of the (converged) warp, the same every time
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// arrive on this barrier of both CTAs when every MMA issued so far has completed
__device__ __forceinline__ void commit2(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// How long L2 is to keep what a load reads.  A row's 512 columns come as keys and, a tile later, as values,
// then no more: keys stay, values and the keys' last 64 columns go first.  128 heads 428 us without the hints,
// 423 with; they also make the room for what is fetched ahead (below).
__device__ __forceinline__ uint64_t l2_first() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t l2_normal() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t l2_last() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// loads into this CTA that complete on a barrier of the pair's first CTA
__device__ __forceinline__ void load_box(uint32_t dst, const void* map, int x, int y, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint "
      "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}
// four blocks of 64 columns (from the block-th on) of the rows from y on
__device__ __forceinline__ void load_blocks(uint32_t dst, const void* map, int y, int block, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint "
      "[%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(map), "r"(0), "r"(y), "r"(block), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void load_rows4(uint32_t dst, const void* map, int x, int r0, int r1, int r2, int r3,
                                           uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
      "l"(map), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(bar), "l"(policy)
      : "memory");
}
// arrive on a barrier of the pair's first CTA, whose MMA thread waits with acquire at the cluster's scope.
// What it announces lies in this CTA's shared memory (or in TMEM, behind a tcgen05 fence), so the release is
// restricted to that: one of all memory (release.cluster on the arrival) waits for every store of the thread,
// 460 us instead of 422 at 128 heads.
__device__ __forceinline__ void arrive_first(uint32_t bar) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  mbar_arrive_remote_relaxed(bar);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two floats as bf16, rounded to nearest: a in the low half
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// ---------------------------------------------------------------- the schedule
// One block lays out the pieces of every pair.  Units in order of requests make an axis, each as long as
// its tiles and kUnitCost for its start; pair k gets the range [k span, (k + 1) span).  A cut never goes
// through the tiles that hold nodes, so that one piece sees all masks.
//
// Where requests have several units and their rows together do not stay in L2, ranges alone would have each
// unit of a request read the rows at another time (16 requests x 16 units x 8192 positions read 2.4 GB
// from memory, not 0.15).  There the units of a request first come as chunks of about `limit` tiles, in
// the order (request, chunk, unit), and are dealt to the pairs one by one, so that neighbouring pairs read
// the same rows at the same time; what is left of the last, unfilled round goes to ranges that even out
// what the dealt chunks left uneven.
constexpr int kPlanThreads = 256;
// Requests that chunks are dealt of: one a thread.  256 requests x 4 units x 2048 positions take 541 us dealt and
// 640 in ranges, so 257 take 647.
constexpr int kDealRequests = 256;
// Tiles (256 rows of 1152 bytes) that stay in L2: 70 MB.  16 units a request x 4400 positions, dealt and in ranges:
// 70 tiles 95 and 81 us, 140 140 and 145, 280 241 and 268, 600 476 and 552.
constexpr int kFarTiles = 240;
constexpr int kWhole = 0x7fffffff;             // `limit` that cuts nothing

struct Request {
  int first, n, cached, tiles, cuts;   // cuts: tiles without nodes, behind each of which a cut may go
  int units, chunks, len;              // chunks of a unit, their tiles (the last one's may differ)
  __device__ __forceinline__ int tasks() const { return units * chunks; }
  __device__ __forceinline__ int cost() const { return len + kUnitCost; }   // of a task
  // where the axis' place v of a unit's tiles may be cut
  __device__ __forceinline__ int cut(int v) const { return v > cuts ? tiles : max(v, 0); }
};
__device__ __forceinline__ Request request_of(const TreeParams& p, int b, int limit = kWhole) {
  Request r;
  r.first = min(max(p.token_start[b], 0), p.T);
  r.n = min(min(max(p.token_start[b + 1], r.first), p.T) - r.first, p.max_nodes);
  r.cached = max(p.cached[b], 0);
  r.tiles = (int)(((long long)r.cached + r.n + kTile - 1) / kTile);
  r.cuts = r.cached / kTile;
  // (cached positions behind the block table: all that there is, the last kernel computes)
  r.units = r.n > 0 && r.cached <= tree_reach(p) ? (r.n * p.h + kRows - 1) / kRows : 0;
  r.chunks = 1;
  r.len = r.tiles;
  if (r.tiles > limit) {
    r.len = (r.tiles + (r.tiles + limit - 1) / limit - 1) / ((r.tiles + limit - 1) / limit);
    r.chunks = min(r.cuts / r.len + 1, (r.tiles + r.len - 1) / r.len);   // none begins behind the last cut
  }
  return r;
}

struct Plan {
  int limit, rounds;                   // chunks dealt: `rounds` to every pair
  int dealt;                           // rounds * pairs
};

// the pieces of one pair, in order: f(request number, request, unit, k0, k1)
template <class Get, class F>
__device__ __forceinline__ void walk_pair(const TreeParams& p, const Plan& plan, const int* tasks_before, Get request,
                                          int pair, int pairs, int b, long long off, long long left, F f) {
  auto piece = [&](int bb, const Request& r, int task, int from, int to) {   // places [from, to) of a task
    const int begin = task / r.units * r.len;
    const bool last = task / r.units == r.chunks - 1;
    const int end = last ? r.tiles : r.cut(begin + r.len);
    const int k0 = max(r.cut(begin + from - kUnitCost), begin);
    const int k1 = to >= r.cost() ? end : min(max(r.cut(begin + to - kUnitCost), begin), end);
    if (k1 > k0) f(bb, r, task % r.units, k0, k1);
  };
  for (int i = 0; i < plan.rounds; ++i) {
    const int t = pair + i * pairs;
    int lo = 0, hi = p.B;                      // the last request with tasks_before <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tasks_before[mid] <= t) lo = mid; else hi = mid;
    }
    const Request r = request(lo);
    piece(lo, r, t - tasks_before[lo], 0, r.cost());
  }
  if (left <= 0) return;
  Request r = request(b);
  auto skipped = [&] { return plan.dealt ? min(max(plan.dealt - tasks_before[b], 0), r.tasks()) : 0; };
  int skip = skipped();
  while (left > 0) {
    if (off >= (long long)(r.tasks() - skip) * r.cost()) {
      if (++b >= p.B) return;
      r = request(b);
      skip = skipped();
      off = 0;
      continue;
    }
    const int c = r.cost();
    const int task = off >> 32 ? (int)(off / c) : (int)((uint32_t)off / (uint32_t)c);   // (64 bits are slow)
    const int u = (int)(off - (long long)task * c);
    const int take = (int)min(left, (long long)(c - u));
    off += take;
    left -= take;
    piece(b, r, skip + task, u, u + take);
  }
}

// the sum over the threads before, the sum of all in `total`
__device__ __forceinline__ long long block_before(long long v, long long* part, long long& total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  long long in = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, in, o);
    if (lane >= o) in += u;
  }
  __syncthreads();
  if (lane == 31) part[warp] = in;
  __syncthreads();
  long long before = in - v, sum = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const long long x = part[w];
    before += w < warp ? x : 0;
    sum += x;
  }
  total = sum;
  return before;
}

__global__ void __launch_bounds__(kPlanThreads) tree_schedule_kernel(const TreeTcParams tp) {
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int kKept = 4;                     // pieces of a pair that its first walk keeps for the second
  __shared__ long long part[kPlanThreads / 32], cost_before[kPlanThreads];
  __shared__ int tasks_before[kDealRequests + 1], load[kMaxPairs + 1], load_all;
  __shared__ long long share_at[kMaxPairs + 1];             // where the pairs' ranges lie
  __shared__ Request requests[kPlanThreads];                // where there is one a thread
  __shared__ Piece kept[kMaxPairs][kKept];
  __shared__ int n_of[3], split_of[3], cost_of[3], tiles_of, far_of;   // whole numbers: the same in any order
  const TreeParams& p = tp.p;
  const int tid = threadIdx.x, lane = tid % 32, pairs = tp.pairs;
  const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(tid * per, p.B), r1 = min(r0 + per, p.B);
  Plan plan{kWhole, 0, 0};
  auto request = [&](int b) { return p.B <= kPlanThreads ? requests[b] : request_of(p, b, plan.limit); };
  if (tid < 3) {
    n_of[tid] = split_of[tid] = cost_of[tid] = 0;
  }
  if (tid == 0) tiles_of = far_of = 0;
  for (int w = tid; w < (p.B + 31) / 32; w += kPlanThreads) tp.ws.marks[w] = 0;
  __syncthreads();
  long long cost = 0;                          // of the units
  long long tiles = 0, far = 0;                // their tiles; tiles of different rows
  for (int b = r0; b < r1; ++b) {
    const Request r = request_of(p, b);
    cost += (long long)r.units * r.cost();
    tiles += (long long)r.units * r.tiles;
    far += r.units > 0 ? r.tiles : 0;
    if (p.B <= kPlanThreads) requests[b] = r;
    if (min(max(p.token_start[b + 1], 0), p.T) - min(max(p.token_start[b], 0), p.T) > p.max_nodes)
      report_status(p.status, kStatusBadTree);
    if (r.n > 0 && r.units == 0) tp.ws.mark(b);
  }
  long long total;
  long long at = block_before(cost, part, total);
  if (p.B <= kDealRequests && total > 2 * kFarTiles && total < (1 << 28)) {   // (32 bits from here on)
    auto add = [&](int v, int* to) {
      v = __reduce_add_sync(0xffffffffu, v);
      if (lane == 0) atomicAdd(to, v);
    };
    add((int)tiles, &tiles_of);                // (both below `total`; with a task's starts and last chunk below 3 times that)
    add((int)far, &far_of);
    __syncthreads();
    // From 1.5 units a request on.  Dealt and in ranges, 8192 positions: 64 requests of 1.25 units 177 and 190 us, of 1.5
    // 203 and 235, of 2 274 and 302; 16 requests of 1.5 units 89 and 74, of 2 106 and 92, of 3 124 and 119, of 6 186 and
    // 210; 2 long ones of 131072 positions 498 and 698.
    if (far_of > kFarTiles && 2 * tiles_of >= 3 * far_of) {
      // Whole units, or chunks that make a round or two; what is not dealt counts a third more (77 units of 7000 positions
      // 137 us so, 144 where it counts as much, 138 where it counts twice; other shapes within 2 %)
      int limits[3] = {kWhole, 0, 0};
      for (int c = 0; c < 3; ++c) {
        if (c > 0) limits[c] = (tiles_of + c * pairs - 1) / (c * pairs);
        int n = 0, split = 0, all = 0;
        if (tid < p.B) {
          const Request r = request_of(p, tid, limits[c]);
          n = r.tasks();
          all = n * r.cost();
          split = r.chunks > 1 ? n : 0;
        }
        add(all, &cost_of[c]);
        add(n, &n_of[c]);
        add(split, &split_of[c]);
      }
      __syncthreads();
      float best = 1e30f;
      for (int c = 0; c < 3; ++c) {
        const int n = n_of[c];
        if (n < pairs || n > (1 << 24) || split_of[c] + 2 * pairs > tp.ws.slots) continue;
        const float done = (float)(n / pairs * pairs) / (float)n, t = (float)cost_of[c] * (done + 1.3f * (1.f - done));
        if (t < best) {
          best = t;
          plan.limit = limits[c];
          plan.rounds = n / pairs;
          plan.dealt = plan.rounds * pairs;
        }
      }
    }
  }
  if (plan.rounds > 0) {
    // tasks before each request (one request a thread at most), what the dealt ones load each pair with
    Request r{};
    if (tid < p.B) requests[tid] = r = request_of(p, tid, plan.limit);
    const int mine = tid < p.B ? r.tasks() : 0;
    long long n;
    const int before = (int)block_before(mine, part, n);
    if (tid < p.B) tasks_before[tid] = before;
    if (tid == 0) tasks_before[p.B] = (int)n;
    if (tid <= pairs) load[tid] = 0;
    if (tid == 0) load_all = 0;
    // the rest of the tasks, in cost
    const int skip = min(max(plan.dealt - before, 0), mine);
    cost = tid < p.B ? (long long)(mine - skip) * r.cost() : 0;
    at = block_before(cost, part, total);
    if (tid < p.B) {
      // tasks lo .. hi - 1 go to the pairs lo, lo + 1, ... (mod pairs): so many times to each, and once more
      // to `more` of them; `load` gets the steps at both ends
      const int lo = min(before, plan.dealt), hi = min(before + mine, plan.dealt), c = r.cost();
      const int times = (hi - lo) / pairs, more = (hi - lo) - times * pairs, k0 = lo % pairs, k1 = k0 + more;
      if (times > 0) atomicAdd(&load_all, times * c);
      if (more > 0) {
        atomicAdd(&load[k0], c);
        atomicAdd(&load[k1 <= pairs ? k1 : k1 - pairs], -c);
        if (k1 > pairs) atomicAdd(&load[0], c);
      }
    }
    __syncthreads();
    if (tid < 32) {
      constexpr int kEach = kMaxPairs / 32;
      int v[kEach], run = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int k = kEach * lane + i;
        run += k < pairs ? load[k] : 0;
        v[i] = run;
      }
      int up = run;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += u;
      }
#pragma unroll
      for (int i = 0; i < kEach; ++i) v[i] += up - run + load_all;
      // Level the pairs: the least level that gives the rest room, among the pairs below it.
      int level, count = pairs, sum = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) sum += kEach * lane + i < pairs ? v[i] : 0;
      sum = __reduce_add_sync(0xffffffffu, sum) + (int)total;
      for (;;) {                               // (each turn leaves out a pair, or ends)
        level = (sum + count - 1) / count;
        int s2 = 0, c2 = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i)
          if (kEach * lane + i < pairs && v[i] < level) {
            ++c2;
            s2 += v[i];
          }
        c2 = __reduce_add_sync(0xffffffffu, c2);
        s2 = __reduce_add_sync(0xffffffffu, s2) + (int)total;
        if (c2 == count || c2 == 0) break;
        sum = s2;
        count = c2;
      }
      int room = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) room += kEach * lane + i < pairs ? max(level - v[i], 0) : 0;
      int in = room;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += u;
      }
      int from = in - room;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int k = kEach * lane + i;
        if (k < pairs) {
          share_at[k] = min(from, (int)total);
          from += max(level - v[i], 0);
        }
      }
      if (lane == 0) share_at[pairs] = total;
    }
  } else {
    const long long span = max(total >> 31 ? (total + pairs - 1) / pairs : (long long)(((uint32_t)total + pairs - 1) / pairs),
                               (long long)kMinSpan);
    if (tid <= pairs) share_at[tid] = min(tid * span, total);
  }
  cost_before[tid] = at;
  __syncthreads();
  // the pairs' pieces: counted, then written
  const bool have = tid < pairs;
  int first = 0;
  long long off = 0, left = 0;
  if (have) {
    const long long from = share_at[tid];
    left = share_at[tid + 1] - from;
    if (left > 0) {                            // its range begins in this request, this far in
      int lo = 0, hi = kPlanThreads;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cost_before[mid] <= from) lo = mid; else hi = mid;
      }
      long long a = cost_before[lo];
      for (int b = lo * per; b < p.B; ++b) {
        const Request r = request(b);
        const int skip = plan.dealt ? min(max(plan.dealt - tasks_before[b], 0), r.tasks()) : 0;
        const long long c = (long long)(r.tasks() - skip) * r.cost();
        first = b;
        off = from - a;
        if (from < a + c) break;
        a += c;
      }
    }
  }
  auto describe = [&](int b, const Request& r, int unit, int k0, int k1) {
    Piece x;
    x.row0 = r.first * p.h + unit * kRows;
    x.rows = min(kRows, r.n * p.h - unit * kRows);
    x.k0 = k0;
    x.k1 = k1;
    x.request = b;
    x.cached = r.cached;
    x.n = r.n;
    x.first = r.first;
    x.slot = k0 == 0 && k1 == r.tiles ? -1 : 0;
    x.alone = r.units == 1;
    x.pad[0] = x.pad[1] = 0;
    return x;
  };
  int pieces = 0, partials = 0;
  if (have)
    walk_pair(p, plan, tasks_before, request, tid, pairs, first, off, left,
              [&](int b, const Request& r, int unit, int k0, int k1) {
                if (pieces < kKept) kept[tid][pieces] = describe(b, r, unit, k0, k1);
                ++pieces;
                partials += !(k0 == 0 && k1 == r.tiles);
              });
  long long all;                               // (both counts in one sum)
  const long long before = block_before((long long)pieces << 32 | partials, part, all);
  int at_piece = (int)(before >> 32), at_partial = (int)(before & 0xffffffff);
  // Requests whose tokens overlap can have more units than the workspace holds pieces: nothing is done then.
  const bool fits = (all >> 32) <= tp.ws.most && (all & 0xffffffff) <= tp.ws.slots;
  if (have) tp.ws.start[tid] = fits ? at_piece : 0;
  if (tid == 0) {
    tp.ws.start[pairs] = fits ? (int)(all >> 32) : 0;
    *tp.ws.partials = fits ? (int)(all & 0xffffffff) : 0;
    if (!fits) report_status(p.status, kStatusBadTree);
  }
  if (!fits) return;
  auto write = [&](Piece x) {
    if (x.slot == 0) {
      x.slot = at_partial;
      tp.ws.list[at_partial++] = Partial{x.row0, x.rows, x.request, x.k0 == 0};
    }
    tp.ws.pieces[at_piece++] = x;
  };
  if (have) {
    if (pieces <= kKept)
      for (int i = 0; i < pieces; ++i) write(kept[tid][i]);
    else
      walk_pair(p, plan, tasks_before, request, tid, pairs, first, off, left,
                [&](int b, const Request& r, int unit, int k0, int k1) { write(describe(b, r, unit, k0, k1)); });
  }
}

// a pair's pieces, one after the other
struct Walk {
  const Piece* at;
  const Piece* end;
  __device__ __forceinline__ bool next(Piece& x) {
    if (at >= end) return false;
    int4* to = reinterpret_cast<int4*>(&x);
    const int4* from = reinterpret_cast<const int4*>(at++);
    to[0] = __ldcg(from);
    to[1] = __ldcg(from + 1);
    to[2] = __ldcg(from + 2);
    return true;
  }
};

// bits [d, d + 64) of the positions that a node attends to, counted from the first node's: all
// before it, its mask among the n nodes, none behind
__device__ __forceinline__ unsigned long long mask_bits(const long long* words, int n_words, int n, int d) {
  auto word = [&](int i) -> unsigned long long {
    if (i < 0) return ~0ull;
    if (i >= n_words || 64 * i >= n) return 0;
    const unsigned long long w = (unsigned long long)words[i];
    return n - 64 * i >= 64 ? w : w & ((1ull << (n - 64 * i)) - 1);
  };
  const int q = d >> 6, r = d & 63;
  const unsigned long long lo = word(q);
  return r == 0 ? lo : lo >> r | word(q + 1) << (64 - r);
}

// kTwo: the weights in two bf16 terms (their rounding, 2^-17, is below fp32 results' needs), else one
template <bool kTwo>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    decode_tree_kernel(const __grid_constant__ CUtensorMap map_box, const __grid_constant__ CUtensorMap map_v,
                       const __grid_constant__ CUtensorMap map_row, const __grid_constant__ CUtensorMap map_q,
                       const TreeTcParams tp) {
  constexpr int kSlots = Ring<kTwo>::kSlots, kOffRing = Ring<kTwo>::kOff;
  const TreeParams& p = tp.p;
  extern __shared__ char smem_raw[];
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint32_t* tmem_s = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_s = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1;
  const long long wl = p.wait_limit;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&bars[kBarFull + s], 1);      // (first CTA) armed for both CTAs' bytes
      mbar_init(&bars[kBarEmpty + s], 1);     // the MMAs that read the slot have completed
    }
    mbar_init(&bars[kBarQFull], 1);           // (first CTA) q of both CTAs
    mbar_init(&bars[kBarS], 1);               // scores of this buffer complete
    mbar_init(&bars[kBarS + 1], 1);
    mbar_init(&bars[kBarP], 2 * kSoftWarps);  // (first CTA) both CTAs' softmax warps: P written, O rescaled
    mbar_init(&bars[kBarPv], 1);              // P V of a tile has completed
    mbar_init(&bars[kBarO], 2 * kSoftWarps);  // (first CTA) the softmax warps have read O
    mbar_init(&bars[kBarMx], 4);              // the four warps of a row have left their values
    mbar_init(&bars[kBarMx + 1], 4);
    mbar_init(&bars[kBarFin], 1);
    mbar_init(&bars[kBarNever], 1);           // nothing arrives: the stall test hook waits on it
    *abort_s = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc2(tmem_s, kTmemCols);
    tmem_relinquish2();
  }
  if (warp == kLoadWarp && lane == 0) {
    prefetch_tmap(&map_box);
    prefetch_tmap(&map_v);
    prefetch_tmap(&map_q);
  }
  asm volatile("griddepcontrol.launch_dependents;");
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_s;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the schedule is there
  const int begin = __ldcg(tp.ws.start + pair), len = __ldcg(tp.ws.start + pair + 1) - begin;
  Walk walk{tp.ws.pieces + begin, tp.ws.pieces + begin + len};
  Piece x;

  auto fail = [&] {
    report_status(p.status, kStatusTimeout);
    *abort_s = 1;
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa((const void*)abort_s, rank ^ 1u)), "r"(1) : "memory");
  };
  // Waits of a whole warp.  Every branch goes by a vote, which the compiler knows to be the same in all
  // lanes: what is carried through the loops around a wait then stays in uniform registers, which the MMAs
  // and loads take their operands from (with a wait that each lane leaves for itself four MMAs took the
  // issuing warp 480 cycles, now 256, which is their own time).
  auto all = [](bool c) { return __all_sync(0xffffffffu, c) != 0; };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (all(mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = globaltimer_ns();
    for (long long i = 1; i < wl; ++i) {
      if (all(mbar_try_wait(bar, parity))) return true;
      if ((i & 255) == 0 && all(globaltimer_ns() - t0 > 4000000000ull)) return false;
    }
    return false;
  };
  auto aborted = [&] { return __any_sync(0xffffffffu, *abort_s) != 0; };

  if (warp < kSoftWarps) {
    // =================== softmax, rescaling, output =================================
    // Four threads a row: TMEM lane r + 64 half holds the row's scores of keys [128 half, +128), of which
    // warps 0-3 take the first 64 and warps 4-7 the others; they rescale and write the first or the
    // second 128 of the lane's 256 columns of O.
    const int tid = threadIdx.x, lane4 = tid & 127, r = lane4 & 63, half = lane4 >> 6, part = warp >> 2;
    const int row = kHalf * (int)rank + r;                        // of the unit
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t p_ready = mapa(&bars[kBarP], 0), o_read = mapa(&bars[kBarO], 0);
    float* mx = reinterpret_cast<float*>(smem + kOffMx);
    const float c_scale = p.scale * kLog2e;
    // masked scores are -inf, and -inf times a zero scale would be NaN: any valid score times 1e-30
    // still has weight 1
    const float c_abs = fmaxf(fabsf(c_scale), 1e-30f);
    int g = 0, swaps = 0;
    bool ok = true;
    // the values of the three threads with the rest of the row
    auto others = [&](float v, float (&u)[3]) {
      float* at = mx + 256 * (swaps & 1);
      at[tid] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarMx + (warp & 1)]);
      ok = ok && wait_warp(&bars[kBarMx + (warp & 1)], swaps & 1);
      ++swaps;
      u[0] = at[tid ^ 64];
      u[1] = at[tid ^ 128];
      u[2] = at[tid ^ 192];
    };
    // q of a piece: once the piece before has its last scores (the first thread has seen them)
    const uint32_t q_full = mapa(&bars[kBarQFull], 0);
    const uint64_t q_policy = l2_normal();
    auto bring_q = [&](const Piece& y) {
      if (tid != 0) return;
      if (rank == 0) mbar_arrive_expect_tx(&bars[kBarQFull], 2 * kQBytes);
      for (int j = 0; j < 9; ++j)
        load_box(smem_u32(smem + j * kQBlk), &map_q, 64 * j, y.row0 + kHalf * (int)rank, q_full, q_policy);
    };
    Piece y;
    bool more = walk.next(y);
    if (more) bring_q(y);
    while (ok && more) {
      x = y;
      // The sums of the weights as they are, for lse, and as P's one term holds them: out is divided by the
      // latter, so that the rounding of a row's heaviest weights cancels (with two terms 2^-17 of them is left, and
      // the second sum costs 1 to 2 % for 3 to 8 % of the error).  128 heads 414-416 us without the second sum, 419 with,
      // 423 where it came before the hand-over of P.
      float m_ref = -INFINITY, l_sum = 0.f, l_held = 0.f, u[3];
      const bool live = row < x.rows;
      const int node = live ? (x.row0 + row) / p.h - x.first : 0;
      const long long* words = p.mask + (size_t)(x.first + node) * p.words;
      for (int k = x.k0; k < x.k1; ++k, ++g) {
        const int bb = g & 1;
        if (!(ok = !aborted() && wait_warp(&bars[kBarS + bb], (g >> 1) & 1))) break;
        tc_fence_after();
        float s[64];
        {
          uint32_t v[2][32];
          tmem_ld32(lanes + kColS + 128 * bb + 64 * part, v[0]);
          tmem_ld32(lanes + kColS + 128 * bb + 64 * part + 32, v[1]);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 64; ++j) s[j] = __uint_as_float(v[j >> 5][j & 31]);
        }
        if (c_scale < 0.f) {
#pragma unroll
          for (int j = 0; j < 64; ++j) s[j] = -s[j];
        }
        if (k >= x.cached / kTile) {           // a tile with nodes, or with the end
          const int d = (int)((long long)k * kTile + 128 * half + 64 * part - x.cached);
          unsigned long long see = ~0ull;
          if (live) see = mask_bits(words, p.words, x.n, d);
          bool bad = false;
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (!(see >> j & 1)) {
              bad |= !(fabsf(s[j]) <= 3.0e38f);   // (rows behind the end are zeros)
              s[j] = -INFINITY;
            }
          if (bad) tp.ws.mark(x.request);
        }
        float t[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) t[j] = fmaxf(fmaxf(s[j], s[j + 16]), fmaxf(s[j + 32], s[j + 48]));
#pragma unroll
        for (int w = 8; w > 0; w >>= 1)
#pragma unroll
          for (int j = 0; j < w; ++j) t[j] = fmaxf(t[j], t[j + w]);
        others(t[0], u);
        if (!ok) break;
        const float mt = fmaxf(fmaxf(t[0], u[0]), fmaxf(u[1], u[2])) * c_abs;
        float m_new = m_ref;
        if (mt > m_ref + kRescaleThreshold || m_ref == -INFINITY) m_new = fmaxf(mt, m_ref);
        const float base = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = m_ref == m_new ? 1.f : ex2(m_ref - base);
        const bool first = k == x.k0;
        m_ref = m_new;
        float2 sum[2] = {};
        uint32_t pk[32], pl[kTwo ? 32 : 1];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float e0 = ex2(fmaf(s[2 * j], c_abs, -base)), e1 = ex2(fmaf(s[2 * j + 1], c_abs, -base));
          sum[j & 1] = add2(sum[j & 1], make_float2(e0, e1));
          pk[j] = pack_bf16(e0, e1);
          if (kTwo) pl[j] = pack_bf16(e0 - __uint_as_float(pk[j] << 16), e1 - __uint_as_float(pk[j] & 0xffff0000u));
        }
        l_sum = l_sum * alpha + ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
        // P's place and O are free once P V of the tile before has completed
        if (g > 0) {
          if (!(ok = wait_warp(&bars[kBarPv], (g - 1) & 1))) break;
          tc_fence_after();
        }
        char* pb = smem + kOffP + (2 * half + part) * kQBlk + r * 128;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          *reinterpret_cast<uint4*>(pb + ((j ^ (r & 7)) * 16)) =
              make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
          if (kTwo)
            *reinterpret_cast<uint4*>(pb + kPBytes + ((j ^ (r & 7)) * 16)) =
                make_uint4(pl[4 * j], pl[4 * j + 1], pl[4 * j + 2], pl[4 * j + 3]);
        }
        fence_proxy_async_smem();
        if (!first && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (int c = 128 * part; c < 128 * part + 128; c += 32) {
            uint32_t o[32];
            tmem_ld32(lanes + kColO + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
            tmem_st16(lanes + kColO + c, *reinterpret_cast<const uint32_t(*)[16]>(&o[0]));
            tmem_st16(lanes + kColO + c + 16, *reinterpret_cast<const uint32_t(*)[16]>(&o[16]));
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(p_ready);
        if (!kTwo) {                           // (behind the hand-over, beside the MMAs)
          float2 held[2] = {};
#pragma unroll
          for (int j = 0; j < 32; ++j)
            held[j & 1] = add2(held[j & 1], make_float2(__uint_as_float(pk[j] << 16), __uint_as_float(pk[j] & 0xffff0000u)));
          l_held = l_held * alpha + ((held[0].x + held[0].y) + (held[1].x + held[1].y));
        }
      }
      if (!ok) break;
      more = walk.next(y);
      if (more) bring_q(y);
      // ---- the piece's result
      others(l_sum, u);
      const float l = (l_sum + u[0]) + (u[1] + u[2]);
      float l_of_p = l;
      if (!kTwo) {
        others(l_held, u);
        l_of_p = (l_held + u[0]) + (u[1] + u[2]);
      }
      if (!ok || !(ok = wait_warp(&bars[kBarPv], (g - 1) & 1))) break;
      tc_fence_after();
      const bool none = l == 0.f;
      const float inv = none ? 0.f : 1.f / l_of_p;
      const float lse = none ? -INFINITY : (m_ref + __log2f(l)) * kLn2;
      const bool whole = x.slot < 0;
      // A warp's 32 rows go through its own 4 KB of P, 128 bytes a row at a time, so that eight lanes write
      // a row's 128 bytes (a row a lane, 16 bytes a store, took 17000 cycles a piece)
      const bool as16 = whole && p.out_bf16;
      char* stage = smem + kOffP + (2 * half + part) * kQBlk + (warp & 1) * 32 * 128;
      const int row0 = kHalf * (int)rank + (warp & 1) * 32;         // the warp's first row
      char* to = whole ? static_cast<char*>(p.out) + (size_t)(x.row0 + row0) * kDV * (as16 ? 2 : 4)
                       : reinterpret_cast<char*>(tp.ws.part + ((size_t)x.slot * tp.ws.cap + row0) * kDV);
      const int pitch = kDV * (as16 ? 2 : 4), left = x.rows - row0;
      to += (256 * half + 128 * part) * (as16 ? 2 : 4);
      const int wide = as16 ? 64 : 32;                              // columns of 128 bytes
#pragma unroll 1
      for (int c = 0; c < 128; c += wide) {
        uint32_t o[32];
        tmem_ld32(lanes + kColO + 128 * part + c, o);
        tmem_ld_wait();
        if (as16) {
          uint32_t o2[32];
          tmem_ld32(lanes + kColO + 128 * part + c + 32, o2);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            o[j] = pack_bf16(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            o[16 + j] = pack_bf16(__uint_as_float(o2[2 * j]) * inv, __uint_as_float(o2[2 * j + 1]) * inv);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * inv);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((j ^ (lane & 7)) * 16)) =
              make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = 4 * i + (lane >> 3);
          const uint4 y = *reinterpret_cast<const uint4*>(stage + rr * 128 + (((lane & 7) ^ (rr & 7)) * 16));
          if (rr < left) *reinterpret_cast<uint4*>(to + (size_t)rr * pitch + c * (as16 ? 2 : 4) + (lane & 7) * 16) = y;
        }
        __syncwarp();
      }
      if (live && half == 0 && part == 0) {
        if (whole) p.lse[x.row0 + row] = lse;
        else tp.ws.lse[(size_t)x.slot * tp.ws.cap + row] = lse;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_first(o_read);
    }
    if (!ok) fail();
  } else if (warp == kMmaWarp && rank == 0) {
    // =================== MMAs =========================================================
    // One elected lane, the waits included: in a region of one lane the operands stay in uniform registers
    // and four MMAs take it 267 cycles, their own time being 256 (a lane chosen by its number 375; a warp
    // whose lanes all wait, with the MMAs elected, 480).
    if (rank == 0 && len > 0 && elect_one()) {
      const uint32_t id_qk = idesc_bf16(128, 256, 0, 0), id_pv = idesc_bf16(128, 256, 0, 1);
      const uint32_t sm0 = smem_u32(smem);
      const uint32_t dq = desc_lo(sm0, 16), dp = desc_lo(sm0 + kOffP, 16);
      const uint32_t dk = desc_lo(sm0 + kOffRing, 16), dv = desc_lo(sm0 + kOffRing, 4096);
      int slot = 0, g = 0, pieces = 0;
      uint32_t round = 0;
      // test hook: a wait that cannot complete, so the wait limit runs out
      bool ok = !p.stall || mbar_wait(&bars[kBarNever], 0, wl);
      auto qk = [&](int tile) {                // scores of the tile-th tile of all
        const uint32_t d = tmem + kColS + 128 * (tile & 1);
#pragma unroll 1
        for (int j = 0; j < kKChunks; ++j) {
          ok = ok && mbar_wait(&bars[kBarFull + slot], round, wl);
          if (!ok) return;
          tc_fence_after();
          const uint32_t a = dq + j * (kQBlk >> 4), b = dk + slot * (kChunk >> 4);
#pragma unroll
          for (int u = 0; u < 4; ++u) mma2(d, a + 2 * u, b + 2 * u, id_qk, j > 0 || u > 0);
          commit2(&bars[kBarEmpty + slot]);
          if (++slot == kSlots) {
            slot = 0;
            round ^= 1;
          }
        }
        commit2(&bars[kBarS + (tile & 1)]);
      };
      while (ok && walk.next(x)) {
        if (!(ok = mbar_wait(&bars[kBarQFull], pieces & 1, wl))) break;
        tc_fence_after();
        qk(g);
        for (int k = x.k0; ok && k < x.k1; ++k, ++g) {
          if (k + 1 < x.k1) qk(g + 1);
          if (*abort_s) ok = false;
          ok = ok && mbar_wait<true>(&bars[kBarP], g & 1, wl);
          const bool begin = k == x.k0;
          if (begin && pieces > 0) ok = ok && mbar_wait<true>(&bars[kBarO], (pieces - 1) & 1, wl);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int j = 0; j < kVChunks; ++j) {
            ok = ok && mbar_wait(&bars[kBarFull + slot], round, wl);
            if (!ok) break;
            tc_fence_after();
            // 32 keys, all of the CTA's columns: two steps of 16 keys, both halves of O with one P
            const uint32_t a = dp + (j >> 1) * (kQBlk >> 4) + (j & 1) * 4, b = dv + slot * (kChunk >> 4);
            const uint32_t d = tmem + kColO;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              mma2_pair(d, d + 128, a + 2 * u, b + 128 * u, b + 512 + 128 * u, id_pv, !begin || j > 0 || u > 0);
              if (kTwo) mma2_pair(d, d + 128, a + (kPBytes >> 4) + 2 * u, b + 128 * u, b + 512 + 128 * u, id_pv, 1);
            }
            commit2(&bars[kBarEmpty + slot]);
            if (++slot == kSlots) {
              slot = 0;
              round ^= 1;
            }
          }
          commit2(&bars[kBarPv]);
        }
        ++pieces;
      }
      // the second CTA's last arrivals here: no one else waits for them
      if (ok && pieces > 0) ok = mbar_wait<true>(&bars[kBarO], (pieces - 1) & 1, wl);
      if (!ok) fail();
      commit2(&bars[kBarFin]);
    }
    __syncwarp();
    // Every MMA has completed, and every arrival that commits send to either CTA has landed, before
    // TMEM and shared memory go away: an arrival at a CTA that has ended is a fault.
    if (len > 0 && !__all_sync(0xffffffffu, mbar_wait<true>(&bars[kBarFin], 0, kDrainLimit)))
      report_status(p.status, kStatusTimeout);
  } else if (warp >= kLoadWarp && warp < kLoadWarp + kSlots) {
    // =================== keys and values ============================================
    // Warp s fills slot s of the ring, every kSlots-th chunk of the order: it works out where its next chunk
    // lies while it waits for the slot, so a slot is asked for again ~200 cycles after it was read (four
    // warps that took chunks by turns: 400 to 1000).  Each waits for every round of its slot, so that a wait
    // by parity cannot take an older round for its own.
    const int slot = warp - kLoadWarp;
    const int k_step = tp.box ? tp.box : 4, v_step = min(k_step, 32), v_boxes = 32 / v_step;
    const uint32_t full = mapa(&bars[kBarFull + slot], 0), dst = smem_u32(smem + kOffRing + slot * kChunk);
    bool ok = true, bad = false;
    const uint64_t keep = l2_last(), drop = l2_first();
    int round = 0, group = 0, r = slot;        // r-th chunk of the piece's group (K or V of a tile)
    // no block for the positions [pos, pos + n): that matters where a node attends to one of them
    auto missed = [&](int pos, int n) {
      for (int u = 0; u < n && !bad; ++u) {
        const int j = pos + u - x.cached;
        if (j < 0) bad = true;
        for (int i = 0; i < x.n && j >= 0 && !bad; ++i)
          bad = p.mask[(size_t)(x.first + i) * p.words + j / 64] >> (j % 64) & 1;
      }
    };
    bool more = walk.next(x);
    while (more) {
      // groups of a piece of t tiles: K(0), K(1), V(0), ..., K(t - 1), V(t - 2), V(t - 1)
      const int t = x.k1 - x.k0;
      const bool is_k = group == 0 || ((group & 1) && group < 2 * t - 1);
      const int count = is_k ? kKChunks : kVChunks;
      if (r >= count) {
        r -= count;
        if (++group == 2 * t) {
          if (bad) tp.ws.mark(x.request);
          bad = false;
          group = 0;
          more = walk.next(x);
        }
        continue;
      }
      const int tile = x.k0 + (is_k ? (group + 1) / 2 : group == 2 * t - 1 ? t - 1 : group / 2 - 1);
      // the lane's box: `step` rows from `pos` on, 64 columns; of V, with boxes of 32 rows, one lane brings
      // the four blocks of columns
      const int step = is_k ? k_step : v_step;
      const int boxes = is_k ? 128 / k_step : v_boxes == 1 ? 1 : 4 * v_boxes;
      const int at = (is_k ? lane : lane % v_boxes) * step;
      const long long pos = (long long)tile * kTile + (is_k ? 128 * (int)rank : 32 * r) + at;
      const int col = is_k ? 64 * r : 256 * (int)rank + 64 * (lane / v_boxes);
      const uint32_t to = dst + (is_k ? 0 : lane / v_boxes * 4096) + at * 128;
      const int n = lane < boxes ? (int)min(max((long long)x.cached + x.n - pos, 0ll), (long long)step) : 0;
      const int32_t* table = p.block_table + (size_t)x.request * p.max_blocks;
      // its cache rows; those that do not exist are the row behind the last, which loads as zeros
      int row[4], have = n;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        row[u] = tp.num_rows;
        if (u == 0 ? n > 0 : !tp.box && u < n) {
          const uint32_t q = (uint32_t)(pos + u), blk = q / (uint32_t)p.block_size;   // (below 2^31 + 256)
          const int phys = blk < (uint32_t)p.max_blocks ? table[blk] : -1;
          if ((uint32_t)phys < (uint32_t)p.num_blocks) {
            row[u] = phys * p.block_size + (int)(q - blk * (uint32_t)p.block_size);
          } else {
            missed((int)(pos + u), tp.box ? n : 1);
            if (tp.box) have = 0;
          }
        }
      }
      const bool cut = __any_sync(0xffffffffu, tp.box && have != 0 && have != step);
      if (round > 0 && (aborted() || !wait_warp(&bars[kBarEmpty + slot], (round - 1) & 1))) {
        ok = false;
        break;
      }
      if (rank == 0) {
        if (lane == 0) mbar_arrive_expect_tx(&bars[kBarFull + slot], 2 * kChunk);
        __syncwarp();
      }
      // every lane with a box in one instruction (a loop over an elected lane's took half as long again);
      // where the sequence ends in a box, its rows four at a time, with zeros behind the end
      const bool four = !is_k && v_boxes == 1;
      const uint64_t policy = is_k && r < 8 ? keep : drop;
      if (!tp.box) {
        if (lane < boxes) load_rows4(to, &map_row, col, row[0], row[1], row[2], row[3], full, policy);
      } else if (!cut) {
        if (four) {
          if (lane == 0) load_blocks(to, &map_v, row[0], col / 64, full, policy);
        } else if (lane < boxes) {
          load_box(to, &map_box, col, row[0], full, policy);
        }
      } else {
        const bool whole = have == 0 || have == step;
        if (lane < boxes && whole) {
          if (four) load_blocks(to, &map_v, row[0], col / 64, full, policy); else load_box(to, &map_box, col, row[0], full, policy);
        }
        __syncwarp();
        for (int c = 0; c < (four ? 4 : 1); ++c)
          for (int a = 0; a < step; a += 4) {
            auto row_at = [&](int u) { return a + u < have ? row[0] + a + u : tp.num_rows; };
            if (lane < boxes && !whole)
              load_rows4(to + c * 4096 + a * 128, &map_row, col + 64 * c, row_at(0), row_at(1), row_at(2), row_at(3), full, policy);
            __syncwarp();
          }
      }
      __syncwarp();
      ++round;
      r += kSlots;
    }
    if (!ok) fail();
  } else if (warp == kMmaWarp) {
    // =================== rows fetched ahead ============================================
    // The second CTA's warp has no MMAs: it fetches rows that only this pair reads into L2, once a tile's
    // scores are there those of the tile after the next (of the next as well where a piece begins).  The
    // ring alone has too few loads under way for memory's latency: 64 x 8 nodes x 16 heads, bf16 results,
    // 183 us without and 165 with.  Three tiles ahead 183: L2 then loses rows before they are read.  In a
    // steady trickle, a line a time: with nine lines of a row at once 170.
    int g = 0;
    bool ok = true;
    while (ok && walk.next(x)) {
      const int32_t* table = p.block_table + (size_t)x.request * p.max_blocks;
      for (int k = x.k0; ok && k < x.k1; ++k, ++g) {
        if (!x.alone) continue;
        for (int next = k == x.k0 ? k + 1 : k + 2; next <= k + 2; ++next) {
          // (a warp that is a round of the barrier behind would wait for the next: the end ends it)
          bool there = next < k + 2;
          for (long long i = 0; i < wl && ok && !there; ++i) {
            there = all(mbar_try_wait(&bars[kBarS + (g & 1)], (g >> 1) & 1));
            ok = there || !(aborted() || all(mbar_try_wait(&bars[kBarFin], 0)));
          }
          ok = ok && there;
          if (!ok || next >= x.k1) break;
#pragma unroll 1
          for (int u = 0; u < kTile / 32; ++u) {
            const uint32_t q = (uint32_t)next * kTile + 32 * u + lane, blk = q / (uint32_t)p.block_size;
            const int phys = blk < (uint32_t)p.max_blocks && q < (uint32_t)x.cached + x.n ? table[blk] : -1;
            if ((uint32_t)phys < (uint32_t)p.num_blocks) {
              const char* at = reinterpret_cast<const char*>(p.kv) +
                               ((size_t)phys * p.block_size + (q - blk * (uint32_t)p.block_size)) * (2 * kDQK);
#pragma unroll 1
              for (int c = 0; c < 9; ++c) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + 128 * c));
            }
            __syncwarp();
          }
        }
      }
    }
    // the arrivals at this CTA's barriers have landed, as above
    if (len > 0 && !__all_sync(0xffffffffu, mbar_wait<true>(&bars[kBarFin], 0, kDrainLimit)))
      report_status(p.status, kStatusTimeout);
  }

  // ---- teardown
  __syncwarp();
  __syncthreads();
  if (threadIdx.x == 0) {
    if (*abort_s) {
      // loads of either CTA may be in flight: they land within microseconds
      const uint64_t t0 = globaltimer_ns();
      for (int i = 0; i < (1 << 20) && globaltimer_ns() - t0 < 2000000ull; ++i) __nanosleep(1000);
    }
  }
  __syncthreads();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 0) tmem_dealloc2(tmem, kTmemCols);
}

// ---------------------------------------------------------------- joining, and the marked requests
constexpr int kJoinThreads = 128;
constexpr int kFixHeads = 2;

// Every block takes a run of the cut units' rows.
__global__ void __launch_bounds__(kJoinThreads) join_tree_kernel(const TreeTcParams tp) {
  extern __shared__ float smem_f[];
  __shared__ int slots[kMaxSlots];             // a unit's parts
  __shared__ int begins[kMaxSlots], rows_before[kMaxSlots + 1];   // partial results that begin a unit
  __shared__ int sums[kJoinThreads / 32], n_parts;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const TreeParams& p = tp.p;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int partials = min(*tp.ws.partials, tp.ws.slots);
  int any = 0;
  const int words = (p.B + 31) / 32;
  for (int w = tid; w < words; w += kJoinThreads) any |= tp.ws.marks[w] != 0;
  any = __syncthreads_or(any);
  int n_begins = 0, n_rows = 0;
  for (int j0 = 0; j0 < partials; j0 += kJoinThreads) {
    const int j = j0 + tid;
    const Partial x = j < partials ? tp.ws.list[j] : Partial{0, 0, 0, 0};
    const int v = x.begins ? x.rows | 1 << 16 : 0;   // rows (at most 128 x 128 of a round) and a count
    int in = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += u;
    }
    if (lane == 31) sums[warp] = in;
    __syncthreads();
    int before = in - v, all = 0;
    for (int w = 0; w < kJoinThreads / 32; ++w) {
      if (w < warp) before += sums[w];
      all += sums[w];
    }
    if (x.begins) {
      begins[n_begins + (before >> 16)] = j;
      rows_before[n_begins + (before >> 16)] = n_rows + (before & 0xffff);
    }
    n_begins += all >> 16;
    n_rows += all & 0xffff;
    __syncthreads();
  }
  // a row a warp; a block's rows lie next to each other, so that they mostly are of one unit
  constexpr int kWarps = kJoinThreads / 32;
  int unit = -1, n = 0;
  const int run = (n_rows + gridDim.x - 1) / gridDim.x, to = min((int)(blockIdx.x + 1) * run, n_rows);
  for (int it0 = blockIdx.x * run; it0 < to;) {
    int lo = 0, hi = n_begins;                 // the last unit that begins with this row or before
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (rows_before[mid] <= it0) lo = mid; else hi = mid;
    }
    const Partial me = tp.ws.list[begins[lo]];
    const int end = min(to, rows_before[lo] + me.rows);
    if (lo != unit) {                          // its parts, in the order of the slots: the same sums every time
      unit = lo;
      __syncthreads();
      if (warp == 0) {
        int k = 0;
        for (int j0 = 0; j0 < partials; j0 += 32) {
          const bool one = j0 + lane < partials && tp.ws.list[j0 + lane].row0 == me.row0;
          const unsigned m = __ballot_sync(0xffffffffu, one);
          if (one) slots[k + __popc(m & ((1u << lane) - 1))] = j0 + lane;
          k += __popc(m);
        }
        if (lane == 0) n_parts = k;
      }
      __syncthreads();
      n = n_parts;
    }
    const bool skip = any && (tp.ws.marks[me.request / 32] >> (me.request % 32) & 1);   // all of it is computed below
    for (int it = it0 + warp; it < end && !skip; it += kWarps) {
      const int r = it - rows_before[lo];
      if (r >= tp.ws.cap) break;
      const size_t cap = tp.ws.cap;
      const float* lse = tp.ws.lse + r;
      float m = -INFINITY;
      for (int j = lane; j < n; j += 32) m = fmaxf(m, lse[slots[j] * cap]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      float sum = 0.f;
      float4 o[4] = {};
#pragma unroll 2
      for (int j = 0; j < n; ++j) {
        const float l = lse[slots[j] * cap];
        const float e = l == -INFINITY ? 0.f : __expf(l - m);   // NaN goes on
        const float4* v = reinterpret_cast<const float4*>(tp.ws.part + (slots[j] * cap + r) * kDV) + lane;
        sum += e;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float4 y = v[32 * c];
          o[c].x += e * y.x; o[c].y += e * y.y; o[c].z += e * y.z; o[c].w += e * y.w;
        }
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const size_t row = (size_t)me.row0 + r;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const size_t at = row * kDV + 4 * (lane + 32 * c);
        if (p.out_bf16)
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
              make_uint2(pack_bf16(o[c].x * inv, o[c].y * inv), pack_bf16(o[c].z * inv, o[c].w * inv));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) =
              make_float4(o[c].x * inv, o[c].y * inv, o[c].z * inv, o[c].w * inv);
      }
      if (lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : m + logf(sum);
    }
    it0 = end;
  }
  if (!any) return;
  // rare: the nodes of every marked request, a node and two heads at a time
  const int groups = (p.h + kFixHeads - 1) / kFixHeads, all = gridDim.x;
  int first = blockIdx.x;                      // the block's next item, counted from the request's first
  for (int w = 0; w < words; ++w)
    for (unsigned m = tp.ws.marks[w]; m; m &= m - 1) {
      const Request r = request_of(p, 32 * w + __ffs(m) - 1);
      const int items = r.n * groups;
      for (; first < items; first += all) tree_simt<kFixHeads>(p, r.first + first / groups, first % groups * kFixHeads, smem_f);
      first -= items;
    }
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

int pairs_of_device() {
  const int n = device_sm_count() / 2;
  return n < 1 ? 1 : n > kMaxPairs ? kMaxPairs : n;
}

long long units_at_most(int B, int T, int h) { return (long long)T * h / kRows + B; }

// places of the workspace's parts; returns its size
size_t lay_out(char* base, int pairs, int B, int T, int h, Workspace& ws) {
  size_t at = 0;
  auto part = [&](size_t bytes) {
    char* q = base + at;
    at += round256(bytes);
    return q;
  };
  const long long rows = (long long)T * h;
  ws.cap = rows < kRows ? (int)rows : kRows;
  // ranges: two cut units a pair; dealt chunks as many again, where there can be several units of a request
  ws.slots = (rows > kRows ? 4 : 2) * pairs;
  ws.most = (int)(units_at_most(B, T, h) + 2 * ws.slots);
  ws.pieces = reinterpret_cast<Piece*>(part((size_t)ws.most * sizeof(Piece)));
  ws.start = reinterpret_cast<int*>(part((size_t)(pairs + 1) * 4));
  ws.partials = reinterpret_cast<int*>(part(4));
  ws.list = reinterpret_cast<Partial*>(part((size_t)ws.slots * sizeof(Partial)));
  ws.part = reinterpret_cast<float*>(part((size_t)ws.slots * ws.cap * kDV * 4));
  ws.lse = reinterpret_cast<float*>(part((size_t)ws.slots * ws.cap * 4));
  ws.marks = reinterpret_cast<unsigned*>(part((size_t)((B + 31) / 32) * 4));
  return at;
}

// launched early: what it does before griddepcontrol.wait runs beside the end of the kernel before
template <class Kernel, class... Args>
cudaError_t launch_after(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

size_t tree_workspace_bytes(int B, int T, int h) {
  Workspace ws;
  return lay_out(nullptr, pairs_of_device(), B, T, h, ws);
}

cudaError_t launch_decode_tree(const TreeParams& p, cudaStream_t stream) {
  if (p.T == 0 || p.B == 0) return cudaSuccess;
  static std::atomic<bool> attr_set[64];   // per device: set once (a repeat is harmless)
  constexpr int kFixSmem = tree_simt_smem(kFixHeads);
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
    for (auto kernel : {decode_tree_kernel<false>, decode_tree_kernel<true>}) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e != cudaSuccess) return e;
    }
    if (dev >= 0 && dev < 64) attr_set[dev].store(true, std::memory_order_release);
  }
  TreeTcParams tp;
  tp.p = p;
  tp.pairs = pairs_of_device();
  tp.num_rows = p.num_blocks * p.block_size;
  // rows of a box: the largest power of two up to 64 that divides the block size, from 8 on
  tp.box = 64;
  while (p.block_size % tp.box != 0) tp.box /= 2;
  if (tp.box < 8) tp.box = 0;
  lay_out(static_cast<char*>(p.workspace), tp.pairs, p.B, p.T, p.h, tp.ws);
  CUtensorMap box, v, row, q;
  if (!make_rows_map(&box, p.kv, tp.num_rows, tp.box ? tp.box : 8) || !make_rows_map(&row, p.kv, tp.num_rows, 1) ||
      !make_blocks_map(&v, p.kv, tp.num_rows, 32, 4) ||
      !make_rows_map(&q, p.q, (long long)p.T * p.h, kHalf))
    return cudaErrorInvalidValue;
  tree_schedule_kernel<<<1, kPlanThreads, 0, stream>>>(tp);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_after(p.out_bf16 ? decode_tree_kernel<false> : decode_tree_kernel<true>, dim3(2 * tp.pairs), kThreads, kSmem,
                   stream, box, v, row, q, tp);
  if (e != cudaSuccess) return e;
  return launch_after(join_tree_kernel, dim3(12 * device_sm_count()), kJoinThreads, kFixSmem, stream, tp);
}

}  // namespace sfa
