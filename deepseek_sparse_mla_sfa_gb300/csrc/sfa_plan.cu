// sfa_plan.cu -- the step plan: block tables and slot maps built on the GPU from request
// lengths ("RFC: MsModeling 支持 Decode Context Parallel 仿真", 2.1.4.1: block_table
// [requests, max_blk_per_seq] and slot_mapping [total_num_tokens] describe where a step's
// tokens live in the paged latent cache).
//
// With cached length c_b and n_b new tokens, request b holds ceil(c_b / bs) blocks and needs
// ceil((c_b + n_b) / bs); the difference comes from the free list in request order.  Token
// i of the step (request-major) is position c_b + (i - start_b), and its slot is
// block * bs + position % bs.  Everything follows from two prefix sums over the requests
// (tokens and fresh blocks), so there is one launch and no exchange between CTAs: every CTA
// forms both sums itself in shared memory (a few KB that stay in L2) and then takes its
// share of the tokens, finding a token's request by binary search.  A fresh block's id is
// read from the free list, never from the table entry that another CTA writes.
//
// Bound: latency (a launch, one dependent load of the lengths, a scan, one load of the table or the
// free list); a step's outputs are 8 bytes a token.  64 requests of one token take 3.9 us on the
// device, 512 requests of up to 300 tokens 5.5 us.
#include <climits>

#include "sfa_internal.h"

namespace sfa {
namespace {

struct PlanParams {
  const int32_t* cached;
  const int32_t* fresh_tokens;
  int B, block_size;
  int32_t* table;
  int max_blocks;
  const int32_t* free_blocks;
  int num_free;
  const int32_t* taken;
  int num_tokens;
  int32_t *seq_lens, *token_start, *positions, *slots, *taken_out;
  int* status;
};

__device__ __forceinline__ long long warp_inclusive(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
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

__device__ __forceinline__ int blocks_of(long long tokens, int bs, int most) {
  const long long n = (tokens + bs - 1) / bs;
  return n < most ? (int)n : most;
}

template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads) step_plan_kernel(const PlanParams p) {
  constexpr int kPlanWarps = kPlanThreads / 32;
  extern __shared__ int plan_smem[];
  int* tok_s = plan_smem;               // [B + 1] first token of each request
  int* blk_s = plan_smem + p.B + 1;     // [B + 1] fresh blocks of the requests before
  __shared__ long long part_t[kPlanWarps], part_b[kPlanWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);

  long long nt = 0, nb = 0;
  for (int b = b0; b < b1; ++b) {
    const long long c = max(p.cached[b], 0), n = max(p.fresh_tokens[b], 0);
    nt += n;
    nb += blocks_of(c + n, p.block_size, p.max_blocks) - blocks_of(c, p.block_size, p.max_blocks);
  }
  const long long it = warp_inclusive(nt, lane), ib = warp_inclusive(nb, lane);
  if (lane == 31) {
    part_t[warp] = it;
    part_b[warp] = ib;
  }
  __syncthreads();
  long long at = it - nt, ab = ib - nb, total_t = 0, total_b = 0;
  for (int w = 0; w < kPlanWarps; ++w) {
    if (w < warp) {
      at += part_t[w];
      ab += part_b[w];
    }
    total_t += part_t[w];
    total_b += part_b[w];
  }
  for (int b = b0; b < b1; ++b) {
    const long long c = max(p.cached[b], 0), n = max(p.fresh_tokens[b], 0);
    tok_s[b] = (int)min(at, (long long)INT_MAX);
    blk_s[b] = (int)min(ab, (long long)INT_MAX);
    at += n;
    ab += blocks_of(c + n, p.block_size, p.max_blocks) - blocks_of(c, p.block_size, p.max_blocks);
  }
  if (tid == 0) {
    tok_s[p.B] = (int)min(total_t, (long long)INT_MAX);
    blk_s[p.B] = (int)min(total_b, (long long)INT_MAX);
  }
  __syncthreads();

  const int n_tok = tok_s[p.B], n_blk = blk_s[p.B];
  const long long head = max(*p.taken, 0);
  bool bad = false, none = false;
  const int gid = blockIdx.x * kPlanThreads + tid, gsize = gridDim.x * kPlanThreads;

  for (int i = gid; i < p.num_tokens; i += gsize) {
    int pos = -1, slot = -1;
    if (i < n_tok) {
      const int b = last_at_most(tok_s, p.B, i);
      const long long c = max(p.cached[b], 0);
      const long long q = c + (i - tok_s[b]);
      pos = q <= INT_MAX ? (int)q : -1;
      const long long blk = q / p.block_size;
      const long long held = (c + p.block_size - 1) / p.block_size;
      if (blk >= p.max_blocks || pos < 0) {
        none = true;
      } else if (blk < held) {
        const long long phys = p.table[(size_t)b * p.max_blocks + blk];
        const long long s = phys * p.block_size + q % p.block_size;
        if (phys < 0 || s > INT_MAX) bad = true; else slot = (int)s;
      } else {
        const long long f = head + blk_s[b] + (blk - held);
        const long long phys = f < p.num_free ? p.free_blocks[f] : -1;
        const long long s = phys * p.block_size + q % p.block_size;
        if (f >= p.num_free) none = true;
        else if (phys < 0 || s > INT_MAX) bad = true;
        else slot = (int)s;
      }
    }
    p.positions[i] = pos;
    p.slots[i] = slot;
  }
  // fresh table entries: the k-th fresh block of the step
  for (int k = gid; k < n_blk; k += gsize) {
    const int b = last_at_most(blk_s, p.B, k);
    const int held = blocks_of(max(p.cached[b], 0), p.block_size, p.max_blocks);
    const long long f = head + k;
    if (f >= p.num_free) none = true;
    p.table[(size_t)b * p.max_blocks + held + (k - blk_s[b])] = f < p.num_free ? p.free_blocks[f] : -1;
  }
  for (int b = gid; b < p.B; b += gsize) {
    const long long len = (long long)max(p.cached[b], 0) + max(p.fresh_tokens[b], 0);
    p.seq_lens[b] = (int)min(len, (long long)INT_MAX);
    p.token_start[b] = tok_s[b];
  }
  if (gid == 0) {
    p.token_start[p.B] = n_tok;
    *p.taken_out = (int)min(head + n_blk, (long long)max((long long)p.num_free, head));
    if (n_tok > p.num_tokens) none = true;
  }
  if (bad) report_status(p.status, kStatusBadBlock);
  if (none) report_status(p.status, kStatusNoBlocks);
}

}  // namespace

cudaError_t launch_step_plan(const int32_t* cached, const int32_t* fresh_tokens, int B, int block_size,
                             int32_t* table, int max_blocks, const int32_t* free_blocks, int num_free,
                             const int32_t* taken, int num_tokens, int32_t* seq_lens, int32_t* token_start,
                             int32_t* positions, int32_t* slots, int32_t* taken_out, int* status,
                             cudaStream_t stream) {
  const PlanParams p{cached, fresh_tokens, B,        block_size,  table,     max_blocks, free_blocks, num_free,
                     taken,  num_tokens,   seq_lens, token_start, positions, slots,      taken_out,   status};
  // Few requests: small blocks and a token a thread (64 requests 3.9 us, by 512 threads 4.4; 512
  // requests of up to 300 tokens 5.5, with four tokens a thread 7.5).  Many: more threads for the
  // sums, and from some thousands on fewer blocks that form them (8192 requests of 20 tokens 24 us,
  // with a token a thread 49; of 256 threads 128; 4096 requests 8.6 with one, 12.0 with four).
  const bool wide = B > 1024;
  const int threads = wide ? 512 : 256, per_block = (B > 4096 ? 4 : 1) * threads, most = 4 * device_sm_count();
  long long blocks = ((long long)num_tokens + per_block - 1) / per_block;
  const int grid = (int)(blocks < 1 ? 1 : blocks > most ? most : blocks);
  const size_t smem = (size_t)(2 * (B + 1)) * 4, fixed = 2 * (512 / 32) * sizeof(long long);   // (part_t, part_b)
  if (smem + fixed > 48 * 1024) {              // what a launch has unasked holds both
    const cudaError_t e = cudaFuncSetAttribute(step_plan_kernel<512>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)(2 * (kPlanMaxRequests + 1) * 4));
    if (e != cudaSuccess) return e;
  }
  if (wide)
    step_plan_kernel<512><<<grid, threads, smem, stream>>>(p);
  else
    step_plan_kernel<256><<<grid, threads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace sfa
