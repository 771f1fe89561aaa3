// sfa_api.cu -- the C ABI of libsfa.so (declared in include/sfa.h): argument
// checks, kernel selection, the per-device status word and the host-buffer
// entry point.  Every step of the computation runs in this library's kernels.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include <climits>

#include "sfa.h"
#include "sfa_internal.h"

namespace {

// Per-device status word written by kernels (first error wins), read and
// cleared by sfa_last_device_status().
__device__ int g_sfa_status;

constexpr int kMaxDevices = 64;
std::mutex g_mu;
int* g_status_ptr[kMaxDevices] = {};
std::atomic<long long> g_wait_limit{0};
std::atomic<int> g_kernel_path{0};  // 0 automatic, 1 CUDA-core only, 2 CTA-pair tcgen05 for every h
std::atomic<int> g_stall{0};        // test hook: kernels first wait on a barrier nothing completes

// 0: CUDA-core kernel, 1: CTA-pair tcgen05 kernel, 2: small-head tcgen05 kernel,
// 3: stacked-half tcgen05 kernel
int kernel_choice(int h, int block_size) {
  const int path = g_kernel_path.load();
  if (path == 1 || !sfa::tc_supports(h, block_size)) return 0;
  if (path == 2) return 1;
  if (sfa::narrow_supports(h)) return 2;
  return sfa::stack_supports(h) ? 3 : 1;
}
constexpr long long kDefaultWaitLimit = 1LL << 26;  // iterations of a bounded device wait

// helper streams of sfa_decode_host, created once per device on first use
constexpr int kHostGroups = 4;
constexpr double kHostPipeMinOutBytes = 4.0 * (1 << 20);   // smaller results: one group
struct HostPipe {
  std::mutex mu;   // one enqueue sequence at a time uses the shared events
  cudaStream_t s[kHostGroups] = {};
  cudaEvent_t start = nullptr, done[kHostGroups] = {};
};
std::mutex g_pipe_mu;
HostPipe* g_pipe[kMaxDevices] = {};
bool g_pipe_failed[kMaxDevices] = {};

HostPipe* host_pipe(int dev) {
  if (dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lk(g_pipe_mu);
  if (g_pipe[dev] || g_pipe_failed[dev]) return g_pipe[dev];
  HostPipe* hp = new HostPipe;
  bool ok = cudaEventCreateWithFlags(&hp->start, cudaEventDisableTiming) == cudaSuccess;
  for (int g = 0; ok && g < kHostGroups; ++g)
    ok = cudaStreamCreateWithFlags(&hp->s[g], cudaStreamNonBlocking) == cudaSuccess &&
         cudaEventCreateWithFlags(&hp->done[g], cudaEventDisableTiming) == cudaSuccess;
  if (!ok) {
    g_pipe_failed[dev] = true;   // fall back to a single group on the caller's stream
    return nullptr;
  }
  g_pipe[dev] = hp;
  return hp;
}

int* status_word(int dev) {
  if (dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_status_ptr[dev]) {
    void* ptr = nullptr;
    if (cudaGetSymbolAddress(&ptr, g_sfa_status) != cudaSuccess) return nullptr;
    g_status_ptr[dev] = static_cast<int*>(ptr);
  }
  return g_status_ptr[dev];
}

// the status word of the current device (null: none)
int* current_status() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess ? status_word(dev) : nullptr;
}

sfa_status done(cudaError_t e) { return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

sfa_status check_decode_args(const void* q, const void* kv, const int32_t* block_table,
                             const int32_t* seq_lens, const int32_t* topk_idx, int B, int Q, int h,
                             int top_k, int num_blocks, int block_size, int max_blocks_per_seq,
                             float scale, int n_splits) {
  if (B < 0 || Q < 1 || top_k < 0 || num_blocks < 1 || block_size < 1 || max_blocks_per_seq < 1 ||
      n_splits < 1 || h < 1 || !isfinite(scale))
    return SFA_ERR_INVALID_ARG;
  if (h > SFA_MAX_HEADS || n_splits > SFA_MAX_SPLITS) return SFA_ERR_UNSUPPORTED;
  if ((long long)B * Q > 0x7fffffffLL) return SFA_ERR_UNSUPPORTED;
  if ((long long)B * Q == 0) return SFA_OK;
  if (!q || !kv || !block_table || !seq_lens || (!topk_idx && top_k > 0)) return SFA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(topk_idx, 4))
    return SFA_ERR_INVALID_ARG;
  return SFA_OK;
}

}  // namespace

// A captured sfa_decode_host step (see include/sfa.h).
struct sfa_host_plan_s {
  cudaGraph_t graph;
  cudaGraphExec_t exec;
};

extern "C" {

const char* sfa_status_string(sfa_status s) {
  switch (s) {
    case SFA_OK: return "SFA_OK";
    case SFA_ERR_INVALID_ARG: return "SFA_ERR_INVALID_ARG";
    case SFA_ERR_UNSUPPORTED: return "SFA_ERR_UNSUPPORTED";
    case SFA_ERR_WORKSPACE: return "SFA_ERR_WORKSPACE";
    case SFA_ERR_CUDA: return "SFA_ERR_CUDA";
    case SFA_ERR_DEVICE_TIMEOUT: return "SFA_ERR_DEVICE_TIMEOUT";
    case SFA_ERR_DEVICE_BAD_BLOCK: return "SFA_ERR_DEVICE_BAD_BLOCK";
    case SFA_ERR_DEVICE_NO_BLOCKS: return "SFA_ERR_DEVICE_NO_BLOCKS";
    case SFA_ERR_DEVICE_BAD_TREE: return "SFA_ERR_DEVICE_BAD_TREE";
  }
  return "SFA_UNKNOWN_STATUS";
}

int sfa_set_kernel_path(int path) {
  if (path < 0 || path > 2) return -1;
  return g_kernel_path.exchange(path);
}

long long sfa_set_wait_limit(long long iterations) {
  return g_wait_limit.exchange(iterations < 0 ? 0 : iterations);
}

int sfa_set_stall_injection(int on) { return g_stall.exchange(on ? 1 : 0); }

size_t sfa_decode_workspace_bytes(int B, int Q, int h, int top_k, int n_splits) {
  if (B <= 0 || Q <= 0 || h <= 0 || top_k < 0 || n_splits < 1) return 0;
  if (g_kernel_path.load() != 0) return 0;
  return sfa::tc_workspace_bytes(B * Q, h, top_k, n_splits);
}

int sfa_decode_launches(int B, int Q, int h, int top_k, int block_size, int n_splits, int merge,
                        int* tensor_core_path) {
  if (B < 0 || Q < 1 || h < 1 || h > SFA_MAX_HEADS || top_k < 0 || block_size < 1 ||
      n_splits < 1 || n_splits > SFA_MAX_SPLITS)
    return -1;
  const int choice = kernel_choice(h, block_size);
  const bool tc = choice != 0;
  if (tensor_core_path) *tensor_core_path = choice;
  if ((long long)B * Q == 0) return 0;
  int n = tc ? sfa::tc_launches(B * Q, h, top_k, n_splits) : 1;
  if (n_splits > 1 && merge) n += 1;
  return n;
}

sfa_status sfa_lse_merge(const float* out_part, const float* lse_part, int n_splits, int rows,
                         int dv, float* out, float* lse, sfa_stream stream) {
  if (n_splits < 1 || rows < 0 || dv < 1) return SFA_ERR_INVALID_ARG;
  if (n_splits > SFA_MAX_SPLITS) return SFA_ERR_UNSUPPORTED;
  if (rows == 0) return SFA_OK;
  if (!out_part || !lse_part || !out || !lse) return SFA_ERR_INVALID_ARG;
  if (!aligned(out_part, 16) || !aligned(out, 16) || !aligned(lse_part, 4) || !aligned(lse, 4))
    return SFA_ERR_INVALID_ARG;
  cudaError_t e = sfa::launch_lse_merge(out_part, lse_part, n_splits, rows, dv, out, 0, lse,
                                        static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

sfa_status sfa_decode(const void* q, const void* kv, const int32_t* block_table,
                      const int32_t* seq_lens, const int32_t* topk_idx, int B, int Q, int h,
                      int top_k, int num_blocks, int block_size, int max_blocks_per_seq,
                      float scale, int n_splits, float* out, float* lse, float* out_part,
                      float* lse_part, void* workspace, size_t workspace_bytes,
                      sfa_stream stream) {
  return sfa_decode_ex(q, kv, block_table, seq_lens, topk_idx, B, Q, h, top_k, num_blocks, block_size,
                       max_blocks_per_seq, scale, n_splits, 0, 0, out, lse, out_part, lse_part, workspace,
                       workspace_bytes, stream);
}

sfa_status sfa_decode_ex(const void* q, const void* kv, const int32_t* block_table, const int32_t* seq_lens,
                         const int32_t* topk_idx, int B, int Q, int h, int top_k, int num_blocks, int block_size,
                         int max_blocks_per_seq, float scale, int n_splits, int interleave_size, int flags,
                         float* out, float* lse, float* out_part, float* lse_part, void* workspace,
                         size_t workspace_bytes, sfa_stream stream) {
  sfa_status st = check_decode_args(q, kv, block_table, seq_lens, topk_idx, B, Q, h, top_k,
                                    num_blocks, block_size, max_blocks_per_seq, scale, n_splits);
  if (st != SFA_OK) return st;
  if (interleave_size < 0 || (flags & ~SFA_BLOCK_TABLE_PER_TOKEN) != 0) return SFA_ERR_INVALID_ARG;
  const int T = B * Q;
  if (T == 0) return SFA_OK;
  const bool merge_after = n_splits > 1 && out && lse;
  if (n_splits == 1) {
    if (!out || !lse || !aligned(out, 16) || !aligned(lse, 4)) return SFA_ERR_INVALID_ARG;
  } else {
    if (!out_part || !lse_part || !aligned(out_part, 16) || !aligned(lse_part, 4))
      return SFA_ERR_INVALID_ARG;
    if ((out && !lse) || (!out && lse)) return SFA_ERR_INVALID_ARG;
    if (merge_after && (!aligned(out, 16) || !aligned(lse, 4))) return SFA_ERR_INVALID_ARG;
  }
  // the workspace is optional: without enough of it the kernels use a schedule that needs none
  const size_t need = sfa_decode_workspace_bytes(B, Q, h, top_k, n_splits);
  if (need == 0 || !workspace || workspace_bytes < need || !aligned(workspace, 256)) {
    workspace = nullptr;
    workspace_bytes = 0;
  }

  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SFA_ERR_CUDA;
  int* status = status_word(dev);
  if (!status) return SFA_ERR_CUDA;

  sfa::DecodeParams p;
  memset(&p, 0, sizeof p);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kv = static_cast<const __nv_bfloat16*>(kv);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.topk_idx = topk_idx;
  p.B = B;
  p.Q = Q;
  p.h = h;
  p.top_k = top_k;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.max_blocks = max_blocks_per_seq;
  p.scale = scale;
  p.n_splits = n_splits;
  p.out = n_splits == 1 ? out : out_part;
  p.lse = n_splits == 1 ? lse : lse_part;
  p.workspace = workspace;
  p.workspace_bytes = workspace_bytes;
  p.status = status;
  const long long wl = g_wait_limit.load();
  p.wait_limit = wl > 0 ? wl : kDefaultWaitLimit;
  p.interleave = interleave_size;
  p.bt_per_token = (flags & SFA_BLOCK_TABLE_PER_TOKEN) ? 1 : 0;
  p.stall = g_stall.load();

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int choice = kernel_choice(h, block_size);
  const bool tc = choice != 0 && sfa::tc_supports_ptrs(q, kv, p.out);
  cudaError_t e = tc ? sfa::launch_decode_tc(p, choice, s) : sfa::launch_decode_simt(p, s);
  if (e != cudaSuccess) return SFA_ERR_CUDA;
  if (merge_after) {
    e = sfa::launch_lse_merge(out_part, lse_part, n_splits, T * h, SFA_D_V, out, 0, lse, s);
    if (e != cudaSuccess) return SFA_ERR_CUDA;
  }
  return SFA_OK;
}

size_t sfa_decode_host_staging_bytes(int B, int Q, int h, int top_k, int max_blocks_per_seq,
                                     int n_splits) {
  if (B < 0 || Q < 1 || h < 1 || top_k < 0 || max_blocks_per_seq < 1 || n_splits < 1) return 0;
  const size_t T = (size_t)B * Q, a = 256;
  size_t n = 0;
  n += round_up(T * h * SFA_D_QK * 2, a);                 // q
  n += round_up((size_t)B * max_blocks_per_seq * 4, a);   // block_table
  n += round_up((size_t)B * 4, a);                        // seq_lens
  n += round_up(T * top_k * 4, a);                        // topk_idx
  n += round_up(T * h * SFA_D_V * 4, a);                  // out
  n += round_up(T * h * 4, a);                            // lse
  if (n_splits > 1) {
    n += round_up((size_t)n_splits * T * h * SFA_D_V * 4, a);  // out_part
    n += round_up((size_t)n_splits * T * h * 4, a);            // lse_part
  }
  n += round_up(sfa_decode_workspace_bytes(B, Q, h, top_k, n_splits), a);
  return n;
}

// The argument checks of sfa_decode_host (SFA_OK also for an empty batch).
static sfa_status check_host_args(const void* q_host, const void* kv, const int32_t* block_table_host,
                                  const int32_t* seq_lens_host, const int32_t* topk_idx_host, int B, int Q, int h,
                                  int top_k, int num_blocks, int block_size, int max_blocks_per_seq, float scale,
                                  int n_splits, const float* out_host, const float* lse_host, const void* staging,
                                  size_t staging_bytes) {
  const sfa_status st = check_decode_args(q_host, kv, block_table_host, seq_lens_host, topk_idx_host, B, Q, h,
                                          top_k, num_blocks, block_size, max_blocks_per_seq, scale, n_splits);
  if (st != SFA_OK || (long long)B * Q == 0) return st;
  if (!out_host || !lse_host) return SFA_ERR_INVALID_ARG;
  const size_t need = sfa_decode_host_staging_bytes(B, Q, h, top_k, max_blocks_per_seq, n_splits);
  if (!staging || staging_bytes < need || !aligned(staging, 256)) return SFA_ERR_WORKSPACE;
  return SFA_OK;
}

sfa_status sfa_decode_host(const void* q_host, const void* kv, const int32_t* block_table_host,
                           const int32_t* seq_lens_host, const int32_t* topk_idx_host, int B,
                           int Q, int h, int top_k, int num_blocks, int block_size,
                           int max_blocks_per_seq, float scale, int n_splits, float* out_host,
                           float* lse_host, void* staging, size_t staging_bytes,
                           sfa_stream stream) {
  sfa_status st = check_host_args(q_host, kv, block_table_host, seq_lens_host, topk_idx_host, B, Q, h, top_k,
                                  num_blocks, block_size, max_blocks_per_seq, scale, n_splits, out_host, lse_host,
                                  staging, staging_bytes);
  if (st != SFA_OK) return st;
  const size_t T = (size_t)B * Q;
  if (T == 0) return SFA_OK;

  char* base = static_cast<char*>(staging);
  size_t off = 0;
  auto carve = [&](size_t bytes) {
    char* p = base + off;
    off += round_up(bytes, 256);
    return p;
  };
  const size_t q_bytes = T * h * SFA_D_QK * 2, bt_bytes = (size_t)B * max_blocks_per_seq * 4,
               sl_bytes = (size_t)B * 4, idx_bytes = T * top_k * 4,
               out_bytes = T * h * SFA_D_V * 4, lse_bytes = T * h * 4;
  void* q_d = carve(q_bytes);
  int32_t* bt_d = reinterpret_cast<int32_t*>(carve(bt_bytes));
  int32_t* sl_d = reinterpret_cast<int32_t*>(carve(sl_bytes));
  int32_t* idx_d = reinterpret_cast<int32_t*>(carve(idx_bytes));
  float* out_d = reinterpret_cast<float*>(carve(out_bytes));
  float* lse_d = reinterpret_cast<float*>(carve(lse_bytes));
  float* op_d = nullptr;
  float* lp_d = nullptr;
  if (n_splits > 1) {
    op_d = reinterpret_cast<float*>(carve((size_t)n_splits * out_bytes));
    lp_d = reinterpret_cast<float*>(carve((size_t)n_splits * lse_bytes));
  }
  const size_t ws_bytes = sfa_decode_workspace_bytes(B, Q, h, top_k, n_splits);
  void* ws_d = ws_bytes ? carve(ws_bytes) : nullptr;

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // A batch large enough to be copy-bound is split into groups of whole sequences, each
  // on its own helper stream forked from `s`: group g's results travel back while later
  // groups are still being copied in or computed, and copies in both directions use
  // separate copy engines.  Each group uses its own slices of the staging buffers.
  int groups = 1;
  HostPipe* hp = nullptr;
  if ((double)out_bytes >= kHostPipeMinOutBytes && B >= 2) {
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess) hp = host_pipe(dev);
    if (hp) groups = B < kHostGroups ? B : kHostGroups;
  }
  // the block table, sequence lengths and index lists go first, whole, on `s`; each
  // group then copies only its q in and its out back, and lse returns in one copy at the end
  if (cudaMemcpyAsync(bt_d, block_table_host, bt_bytes, cudaMemcpyHostToDevice, s) != cudaSuccess ||
      cudaMemcpyAsync(sl_d, seq_lens_host, sl_bytes, cudaMemcpyHostToDevice, s) != cudaSuccess ||
      (idx_bytes && cudaMemcpyAsync(idx_d, topk_idx_host, idx_bytes, cudaMemcpyHostToDevice, s) != cudaSuccess))
    return SFA_ERR_CUDA;
  std::unique_lock<std::mutex> lk;
  if (groups > 1) {
    lk = std::unique_lock<std::mutex>(hp->mu);
    if (cudaEventRecord(hp->start, s) != cudaSuccess) return SFA_ERR_CUDA;
  }
  for (int g = 0; g < groups; ++g) {
    const int b0 = (int)((long long)B * g / groups), b1 = (int)((long long)B * (g + 1) / groups);
    const int Bg = b1 - b0;
    if (Bg == 0) continue;
    cudaStream_t gs = groups > 1 ? hp->s[g] : s;
    if (groups > 1 && cudaStreamWaitEvent(gs, hp->start, 0) != cudaSuccess) return SFA_ERR_CUDA;
    const size_t t0 = (size_t)b0 * Q, Tg = (size_t)Bg * Q;
    const size_t qo = t0 * h * SFA_D_QK * 2, io = t0 * top_k, oo = t0 * h * SFA_D_V, lo = t0 * h;
    const size_t bo = (size_t)b0 * max_blocks_per_seq;
    char* qg = static_cast<char*>(q_d) + qo;
    if (cudaMemcpyAsync(qg, static_cast<const char*>(q_host) + qo, Tg * h * SFA_D_QK * 2,
                        cudaMemcpyHostToDevice, gs) != cudaSuccess)
      return SFA_ERR_CUDA;
    // a group's shard partials are its own [n_splits, Tg, h, ...] block
    float* opg = op_d ? op_d + (size_t)n_splits * oo : nullptr;
    float* lpg = lp_d ? lp_d + (size_t)n_splits * lo : nullptr;
    st = sfa_decode(qg, kv, bt_d + bo, sl_d + b0, idx_d + io, Bg, Q, h, top_k, num_blocks, block_size,
                    max_blocks_per_seq, scale, n_splits, out_d + oo, lse_d + lo, opg, lpg, ws_d, ws_bytes, gs);
    if (st != SFA_OK) return st;
    if (cudaMemcpyAsync(out_host + oo, out_d + oo, Tg * h * SFA_D_V * 4, cudaMemcpyDeviceToHost, gs) !=
        cudaSuccess)
      return SFA_ERR_CUDA;
    if (groups > 1 && (cudaEventRecord(hp->done[g], gs) != cudaSuccess ||
                       cudaStreamWaitEvent(s, hp->done[g], 0) != cudaSuccess))
      return SFA_ERR_CUDA;
  }
  if (cudaMemcpyAsync(lse_host, lse_d, lse_bytes, cudaMemcpyDeviceToHost, s) != cudaSuccess) return SFA_ERR_CUDA;
  return SFA_OK;
}

sfa_status sfa_host_plan_create(const void* q_host, const void* kv, const int32_t* block_table_host,
                                const int32_t* seq_lens_host, const int32_t* topk_idx_host, int B, int Q, int h,
                                int top_k, int num_blocks, int block_size, int max_blocks_per_seq, float scale,
                                int n_splits, float* out_host, float* lse_host, void* staging,
                                size_t staging_bytes, sfa_host_plan* plan) {
  if (!plan) return SFA_ERR_INVALID_ARG;
  *plan = nullptr;
  const sfa_status chk = check_host_args(q_host, kv, block_table_host, seq_lens_host, topk_idx_host, B, Q, h,
                                         top_k, num_blocks, block_size, max_blocks_per_seq, scale, n_splits,
                                         out_host, lse_host, staging, staging_bytes);
  if (chk != SFA_OK) return chk;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SFA_ERR_CUDA;
  // everything that is set up once per device happens here, outside the capture
  if (!status_word(dev)) return SFA_ERR_CUDA;
  host_pipe(dev);
  if (sfa::prepare_decode_tc() != cudaSuccess || sfa::prepare_decode_narrow() != cudaSuccess ||
      sfa::prepare_decode_stack() != cudaSuccess ||
      sfa::prepare_decode_simt() != cudaSuccess)
    return SFA_ERR_CUDA;
  cudaStream_t cs = nullptr;
  if (cudaStreamCreateWithFlags(&cs, cudaStreamNonBlocking) != cudaSuccess) return SFA_ERR_CUDA;
  if (cudaStreamBeginCapture(cs, cudaStreamCaptureModeThreadLocal) != cudaSuccess) {
    cudaStreamDestroy(cs);
    return SFA_ERR_CUDA;
  }
  const sfa_status st = sfa_decode_host(q_host, kv, block_table_host, seq_lens_host, topk_idx_host, B, Q, h, top_k,
                                        num_blocks, block_size, max_blocks_per_seq, scale, n_splits, out_host,
                                        lse_host, staging, staging_bytes, cs);
  cudaGraph_t graph = nullptr;
  const cudaError_t ce = cudaStreamEndCapture(cs, &graph);
  cudaStreamDestroy(cs);
  if (st != SFA_OK || ce != cudaSuccess || !graph) {
    if (graph) cudaGraphDestroy(graph);
    return st != SFA_OK ? st : SFA_ERR_CUDA;
  }
  cudaGraphExec_t exec = nullptr;
  if (cudaGraphInstantiate(&exec, graph, 0) != cudaSuccess) {
    cudaGraphDestroy(graph);
    return SFA_ERR_CUDA;
  }
  *plan = new sfa_host_plan_s{graph, exec};
  return SFA_OK;
}

sfa_status sfa_host_plan_launch(sfa_host_plan plan, sfa_stream stream) {
  if (!plan) return SFA_ERR_INVALID_ARG;
  return cudaGraphLaunch(plan->exec, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

void sfa_host_plan_destroy(sfa_host_plan plan) {
  if (!plan) return;
  cudaGraphExecDestroy(plan->exec);
  cudaGraphDestroy(plan->graph);
  delete plan;
}

sfa_status sfa_uv_proj(const float* out, const void* w_uv, void* y, int T, int h, sfa_stream stream) {
  if (T < 0 || h < 1 || h > 65535) return SFA_ERR_INVALID_ARG;
  if (T == 0) return SFA_OK;
  if (!out || !w_uv || !y || !aligned(out, 16) || !aligned(w_uv, 16) || !aligned(y, 2)) return SFA_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SFA_ERR_CUDA;
  int* status = status_word(dev);
  if (!status) return SFA_ERR_CUDA;
  const long long wl = g_wait_limit.load();
  return sfa::launch_uv_proj(out, w_uv, y, T, h, wl > 0 ? wl : kDefaultWaitLimit, g_stall.load(), status,
                             static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SFA_OK
             : SFA_ERR_CUDA;
}

sfa_status sfa_kv_write(void* kv, long long num_slots, const int32_t* slot_mapping, const void* rows, int T,
                        sfa_stream stream) {
  if (T < 0 || num_slots < 0) return SFA_ERR_INVALID_ARG;
  if (T == 0) return SFA_OK;
  if (!kv || !slot_mapping || !rows || !aligned(kv, 16) || !aligned(rows, 16) || !aligned(slot_mapping, 4))
    return SFA_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SFA_ERR_CUDA;
  int* status = status_word(dev);
  if (!status) return SFA_ERR_CUDA;
  return sfa::launch_kv_write(kv, num_slots, slot_mapping, rows, T, status, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? SFA_OK
             : SFA_ERR_CUDA;
}

static_assert(SFA_TOPK_MAX_S == sfa::kTopkMaxS, "top-k limit of the header and the kernel");

sfa_status sfa_topk(const float* scores, long long row_stride, const int32_t* seq_lens, int B, int Q, int S, int k,
                    int32_t* topk_idx, sfa_stream stream) {
  if (B < 0 || Q < 1 || S < 0 || k < 1 || row_stride < S || row_stride % 4 != 0) return SFA_ERR_INVALID_ARG;
  if ((long long)B * Q > INT_MAX / 8) return SFA_ERR_UNSUPPORTED;
  if (S > sfa::kTopkMaxS) return SFA_ERR_UNSUPPORTED;
  if (B == 0) return SFA_OK;
  if (!topk_idx || !aligned(topk_idx, 4) || (S > 0 && (!scores || !aligned(scores, 16))) ||
      (seq_lens && !aligned(seq_lens, 4)))
    return SFA_ERR_INVALID_ARG;
  return sfa::launch_topk(scores, row_stride, seq_lens, B, Q, S, k, topk_idx, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? SFA_OK
             : SFA_ERR_CUDA;
}

sfa_status sfa_decode_q8(const void* q, const void* kv8, const float* scales, int group, const int32_t* block_table,
                         const int32_t* seq_lens, const int32_t* topk_idx, int B, int Q, int h, int top_k,
                         int num_blocks, int block_size, int max_blocks_per_seq, float scale, int n_splits,
                         int interleave_size, int flags, void* out, float* lse, float* out_part, float* lse_part,
                         sfa_stream stream) {
  sfa_status st = check_decode_args(q, kv8, block_table, seq_lens, topk_idx, B, Q, h, top_k, num_blocks, block_size,
                                    max_blocks_per_seq, scale, n_splits);
  if (st != SFA_OK) return st;
  if (interleave_size < 0 || (flags & ~(SFA_BLOCK_TABLE_PER_TOKEN | SFA_OUT_BF16)) != 0 || group < 1 ||
      block_size % group != 0)
    return SFA_ERR_INVALID_ARG;
  if ((long long)num_blocks * block_size > INT_MAX) return SFA_ERR_UNSUPPORTED;
  const int T = B * Q;
  if (T == 0) return SFA_OK;
  if (!scales || !aligned(scales, 4)) return SFA_ERR_INVALID_ARG;
  const bool merge_after = n_splits > 1 && out && lse;
  if (n_splits == 1) {
    if (!out || !lse) return SFA_ERR_INVALID_ARG;
  } else {
    if (!out_part || !lse_part || !aligned(out_part, 16) || !aligned(lse_part, 4)) return SFA_ERR_INVALID_ARG;
    if ((out && !lse) || (!out && lse)) return SFA_ERR_INVALID_ARG;
  }
  if (out && (!aligned(out, 16) || !aligned(lse, 4))) return SFA_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SFA_ERR_CUDA;
  int* status = status_word(dev);
  if (!status) return SFA_ERR_CUDA;

  sfa::DecodeQ8Params qp;
  memset(&qp, 0, sizeof qp);
  sfa::DecodeParams& p = qp.p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kv = static_cast<const __nv_bfloat16*>(kv8);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.topk_idx = topk_idx;
  p.B = B;
  p.Q = Q;
  p.h = h;
  p.top_k = top_k;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.max_blocks = max_blocks_per_seq;
  p.scale = scale;
  p.n_splits = n_splits;
  p.out = n_splits == 1 ? static_cast<float*>(out) : out_part;
  p.lse = n_splits == 1 ? lse : lse_part;
  p.status = status;
  const long long wl = g_wait_limit.load();
  p.wait_limit = wl > 0 ? wl : kDefaultWaitLimit;
  p.interleave = interleave_size;
  p.bt_per_token = (flags & SFA_BLOCK_TABLE_PER_TOKEN) ? 1 : 0;
  p.stall = g_stall.load();
  qp.scales = scales;
  qp.group = group;
  const int bf16 = (flags & SFA_OUT_BF16) ? 1 : 0;
  qp.out_bf16 = n_splits == 1 ? bf16 : 0;

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // kernel path 1: the CUDA-core kernel, to cross-check; else the tensor cores' (every shape)
  const cudaError_t e = g_kernel_path.load() == 1 ? sfa::launch_decode_q8_simt(qp, s) : sfa::launch_decode_q8(qp, s);
  if (e != cudaSuccess) return SFA_ERR_CUDA;
  if (merge_after &&
      sfa::launch_lse_merge(out_part, lse_part, n_splits, T * h, SFA_D_V, out, bf16, lse, s) != cudaSuccess)
    return SFA_ERR_CUDA;
  return SFA_OK;
}

size_t sfa_kv_write_q8_workspace_bytes(long long num_slots, int group) {
  if (num_slots <= 0 || group <= 1) return 0;
  return (size_t)((num_slots + group - 1) / group) * sfa::kQ8RecordBytes;
}

sfa_status sfa_kv_write_q8(void* kv8, float* scales, long long num_slots, int group, const int32_t* slot_mapping,
                           const void* rows, int T, void* workspace, size_t workspace_bytes, sfa_stream stream) {
  if (T < 0 || num_slots < 0 || group < 1 || num_slots % group != 0) return SFA_ERR_INVALID_ARG;
  if (group > sfa::kQ8MaxWriteGroup) return SFA_ERR_UNSUPPORTED;
  if (T == 0) return SFA_OK;
  if (!kv8 || !scales || !slot_mapping || !rows || !aligned(kv8, 16) || !aligned(rows, 16) ||
      !aligned(slot_mapping, 4) || !aligned(scales, 4))
    return SFA_ERR_INVALID_ARG;
  const size_t need = sfa_kv_write_q8_workspace_bytes(num_slots, group);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return SFA_ERR_WORKSPACE;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SFA_ERR_CUDA;
  int* status = status_word(dev);
  if (!status) return SFA_ERR_CUDA;
  return sfa::launch_kv_write_q8(kv8, scales, num_slots, group, slot_mapping, rows, T, workspace, status,
                                 static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SFA_OK
             : SFA_ERR_CUDA;
}

sfa_status sfa_step_plan(const int32_t* cached_lens, const int32_t* new_lens, int B, int block_size,
                         int32_t* block_table, int max_blocks_per_seq, const int32_t* free_blocks, int num_free,
                         const int32_t* taken, int num_tokens, int32_t* seq_lens, int32_t* token_start,
                         int32_t* positions, int32_t* slot_mapping, int32_t* taken_out, sfa_stream stream) {
  if (B < 0 || block_size < 1 || max_blocks_per_seq < 1 || num_free < 0 || num_tokens < 0) return SFA_ERR_INVALID_ARG;
  if (B > sfa::kPlanMaxRequests) return SFA_ERR_UNSUPPORTED;
  if (!taken || !taken_out || taken == taken_out || !token_start || (num_tokens > 0 && (!positions || !slot_mapping)) ||
      (num_free > 0 && !free_blocks) || (B > 0 && (!cached_lens || !new_lens || !block_table || !seq_lens)))
    return SFA_ERR_INVALID_ARG;
  if (seq_lens && (seq_lens == cached_lens || seq_lens == new_lens)) return SFA_ERR_INVALID_ARG;
  for (const void* ptr : {(const void*)cached_lens, (const void*)new_lens, (const void*)block_table,
                          (const void*)free_blocks, (const void*)taken, (const void*)seq_lens,
                          (const void*)token_start, (const void*)positions, (const void*)slot_mapping,
                          (const void*)taken_out})
    if (!aligned(ptr, 4)) return SFA_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SFA_ERR_CUDA;
  int* status = status_word(dev);
  if (!status) return SFA_ERR_CUDA;
  return sfa::launch_step_plan(cached_lens, new_lens, B, block_size, block_table, max_blocks_per_seq, free_blocks,
                               num_free, taken, num_tokens, seq_lens, token_start, positions, slot_mapping,
                               taken_out, status, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SFA_OK
             : SFA_ERR_CUDA;
}

static_assert(SFA_PLAN_MAX_REQUESTS == sfa::kPlanMaxRequests && SFA_Q8_MAX_WRITE_GROUP == sfa::kQ8MaxWriteGroup,
              "limits of the header and the kernels");

sfa_status sfa_rope(const void* x, long long x_token_stride, long long x_head_stride, void* out,
                    long long out_token_stride, long long out_head_stride, int dtype, int T, int n, int width,
                    int rot_dim, const int32_t* positions, const double* inv_freq, float mscale, int flags,
                    sfa_stream stream) {
  if (T < 0 || n < 1 || width < 1 || rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > width || !isfinite(mscale) ||
      dtype < 0 || dtype > 2 || (flags & ~(SFA_ROPE_INTERLEAVED | SFA_ROPE_INVERSE | SFA_ROPE_COPY_PADDING)) != 0)
    return SFA_ERR_INVALID_ARG;
  if (rot_dim > SFA_ROPE_MAX_DIM) return SFA_ERR_UNSUPPORTED;
  if (T == 0) return SFA_OK;
  const size_t size = dtype == SFA_DTYPE_FP32 ? 4 : 2;
  if (!x || !out || !positions || !inv_freq || !aligned(x, size) || !aligned(out, size) || !aligned(positions, 4) ||
      !aligned(inv_freq, 8))
    return SFA_ERR_INVALID_ARG;
  if (x == out && (x_token_stride != out_token_stride || x_head_stride != out_head_stride))
    return SFA_ERR_INVALID_ARG;
  if ((T > 1 && out_token_stride == 0) || (n > 1 && out_head_stride == 0)) return SFA_ERR_INVALID_ARG;   // rows of out must differ
  return sfa::launch_rope(x, x_token_stride, x_head_stride, out, out_token_stride, out_head_stride, dtype, T, n, width,
                          rot_dim, positions, inv_freq, (flags & SFA_ROPE_INTERLEAVED) ? 1 : 0,
                          (flags & SFA_ROPE_INVERSE) ? 1 : 0, (flags & SFA_ROPE_COPY_PADDING) ? 1 : 0, mscale,
                          static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SFA_OK
             : SFA_ERR_CUDA;
}

static_assert(SFA_TREE_MAX_NODES == sfa::kTreeMaxNodes && SFA_COMPACT_MAX_BLOCKS == sfa::kMaxPoolBlocks,
              "limits of the header and the kernels");

sfa_status sfa_tree_plan(const int32_t* parents, const int32_t* token_start, const int32_t* cached_lens, int B,
                         int num_tokens, int max_nodes, int64_t* mask, int32_t* positions, sfa_stream stream) {
  if (B < 0 || num_tokens < 0 || max_nodes < 1) return SFA_ERR_INVALID_ARG;
  if (max_nodes > SFA_TREE_MAX_NODES) return SFA_ERR_UNSUPPORTED;
  if (!token_start || !aligned(token_start, 4) || (B > 0 && (!cached_lens || !aligned(cached_lens, 4))))
    return SFA_ERR_INVALID_ARG;
  if (num_tokens == 0) return SFA_OK;
  if (!parents || !mask || !positions || !aligned(parents, 4) || !aligned(mask, 8) || !aligned(positions, 4))
    return SFA_ERR_INVALID_ARG;
  int* status = current_status();
  if (!status) return SFA_ERR_CUDA;
  return done(sfa::launch_tree_plan(parents, token_start, cached_lens, B, num_tokens, max_nodes,
                                    reinterpret_cast<long long*>(mask), positions, status,
                                    static_cast<cudaStream_t>(stream)));
}

sfa_status sfa_tree_accept(const int32_t* tokens, const int32_t* targets, const int32_t* parents,
                           const int32_t* token_start, const int32_t* cached_lens, int B, int num_tokens,
                           int max_nodes, int32_t* path, int32_t* accepted, int32_t* next_tokens, int32_t* seq_lens,
                           sfa_stream stream) {
  if (B < 0 || num_tokens < 0 || max_nodes < 1) return SFA_ERR_INVALID_ARG;
  if (max_nodes > SFA_TREE_MAX_NODES) return SFA_ERR_UNSUPPORTED;
  if (B == 0) return SFA_OK;
  if (!token_start || !cached_lens || !path || !accepted || !next_tokens || !seq_lens ||
      (num_tokens > 0 && (!tokens || !targets || !parents)))
    return SFA_ERR_INVALID_ARG;
  for (const int32_t* ptr : {tokens, targets, parents, token_start, cached_lens, (const int32_t*)path,
                             (const int32_t*)accepted, (const int32_t*)next_tokens, (const int32_t*)seq_lens})
    if (!aligned(ptr, 4)) return SFA_ERR_INVALID_ARG;
  int* status = current_status();
  if (!status) return SFA_ERR_CUDA;
  return done(sfa::launch_tree_accept(tokens, targets, parents, token_start, cached_lens, B, num_tokens, max_nodes,
                                      path, accepted, next_tokens, seq_lens, status,
                                      static_cast<cudaStream_t>(stream)));
}

sfa_status sfa_kv_commit(void* kv, int layers, int num_blocks, int block_size, const int32_t* block_table,
                         int max_blocks_per_seq, const int32_t* cached_lens, const int32_t* path,
                         const int32_t* accepted, int B, int max_nodes, sfa_stream stream) {
  if (layers < 0 || num_blocks < 1 || block_size < 1 || max_blocks_per_seq < 1 || B < 0 || max_nodes < 1)
    return SFA_ERR_INVALID_ARG;
  if (max_nodes > SFA_TREE_MAX_NODES) return SFA_ERR_UNSUPPORTED;
  if (B == 0 || layers == 0) return SFA_OK;
  if (!kv || !block_table || !cached_lens || !path || !accepted || !aligned(kv, 16) || !aligned(block_table, 4) ||
      !aligned(cached_lens, 4) || !aligned(path, 4) || !aligned(accepted, 4))
    return SFA_ERR_INVALID_ARG;
  int* status = current_status();
  if (!status) return SFA_ERR_CUDA;
  return done(sfa::launch_kv_commit(kv, layers, num_blocks, block_size, block_table, max_blocks_per_seq, cached_lens,
                                    path, accepted, B, max_nodes, status, static_cast<cudaStream_t>(stream)));
}

sfa_status sfa_decode_tree(const void* q, const void* kv, const int32_t* block_table, const int32_t* cached_lens,
                           const int32_t* token_start, const int64_t* mask, int B, int num_tokens, int h,
                           int max_nodes, int num_blocks, int block_size, int max_blocks_per_seq, float scale,
                           int flags, void* out, float* lse, void* workspace, size_t workspace_bytes,
                           sfa_stream stream) {
  if (B < 0 || num_tokens < 0 || h < 1 || max_nodes < 1 || num_blocks < 1 || block_size < 1 ||
      max_blocks_per_seq < 1 || !isfinite(scale) || (flags & ~SFA_OUT_BF16) != 0)
    return SFA_ERR_INVALID_ARG;
  if (h > SFA_MAX_HEADS || max_nodes > SFA_TREE_MAX_NODES || B > SFA_PLAN_MAX_REQUESTS ||
      (long long)num_blocks * block_size >= INT_MAX || (long long)num_tokens * h >= INT_MAX)
    return SFA_ERR_UNSUPPORTED;
  if (B == 0 || num_tokens == 0) return SFA_OK;
  if (!q || !kv || !block_table || !cached_lens || !token_start || !mask || !out || !lse || !aligned(q, 16) ||
      !aligned(kv, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(block_table, 4) ||
      !aligned(cached_lens, 4) || !aligned(token_start, 4) || !aligned(mask, 8))
    return SFA_ERR_INVALID_ARG;
  if (workspace_bytes < sfa_decode_tree_workspace_bytes(B, num_tokens, h) ||
      (workspace_bytes > 0 && (!workspace || !aligned(workspace, 256))))
    return SFA_ERR_WORKSPACE;
  sfa::TreeParams p;
  memset(&p, 0, sizeof p);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kv = static_cast<const __nv_bfloat16*>(kv);
  p.block_table = block_table;
  p.cached = cached_lens;
  p.token_start = token_start;
  p.mask = reinterpret_cast<const long long*>(mask);
  p.B = B;
  p.T = num_tokens;
  p.h = h;
  p.max_nodes = max_nodes;
  p.words = (max_nodes + 63) / 64;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.max_blocks = max_blocks_per_seq;
  p.scale = scale;
  p.out_bf16 = (flags & SFA_OUT_BF16) ? 1 : 0;
  p.out = out;
  p.lse = lse;
  p.workspace = workspace;
  p.status = current_status();
  if (!p.status) return SFA_ERR_CUDA;
  const long long wl = g_wait_limit.load();
  p.wait_limit = wl > 0 ? wl : kDefaultWaitLimit;
  p.stall = g_stall.load();
  // kernel path 1: the CUDA-core kernel, to cross-check; else the tensor cores'
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return done(g_kernel_path.load() == 1 ? sfa::launch_decode_tree_simt(p, s) : sfa::launch_decode_tree(p, s));
}

size_t sfa_decode_tree_workspace_bytes(int B, int num_tokens, int h) {
  if (B <= 0 || num_tokens <= 0 || h <= 0 || h > SFA_MAX_HEADS) return 0;
  return sfa::tree_workspace_bytes(B, num_tokens, h);
}

sfa_status sfa_blocks_fork(int32_t* block_table, int rows, int max_blocks_per_seq, int32_t* lens, const int32_t* src,
                           const int32_t* dst, int n, int32_t* shares, int num_blocks, const int32_t* free_blocks,
                           int num_free, const int32_t* taken, int block_size, int32_t* copies, int32_t* taken_out,
                           sfa_stream stream) {
  if (rows < 0 || max_blocks_per_seq < 1 || n < 0 || num_blocks < 1 || num_free < 0 || block_size < 1)
    return SFA_ERR_INVALID_ARG;
  if (!taken || !taken_out || taken == taken_out || !shares || (num_free > 0 && !free_blocks) ||
      (rows > 0 && (!block_table || !lens)) || (n > 0 && (!src || !dst || !copies)))
    return SFA_ERR_INVALID_ARG;
  for (const void* ptr : {(const void*)block_table, (const void*)lens, (const void*)src, (const void*)dst,
                          (const void*)shares, (const void*)free_blocks, (const void*)taken, (const void*)copies,
                          (const void*)taken_out})
    if (!aligned(ptr, 4)) return SFA_ERR_INVALID_ARG;
  int* status = current_status();
  if (!status) return SFA_ERR_CUDA;
  return done(sfa::launch_blocks_fork(block_table, rows, max_blocks_per_seq, lens, src, dst, n, shares, num_blocks,
                                      free_blocks, num_free, taken, block_size, copies, taken_out, status,
                                      static_cast<cudaStream_t>(stream)));
}

size_t sfa_blocks_free_workspace_bytes(int rows, int max_blocks_per_seq) {
  if (rows < 1 || max_blocks_per_seq < 1 || rows > SFA_PLAN_MAX_REQUESTS ||
      (long long)rows * max_blocks_per_seq >= (1 << 30))
    return 0;
  return sfa::blocks_free_workspace_bytes(rows, max_blocks_per_seq);
}

sfa_status sfa_blocks_free(const int32_t* block_table, const int32_t* held_lens, const int32_t* keep_lens, int rows,
                           int max_blocks_per_seq, int32_t* shares, int num_blocks, int32_t* free_blocks,
                           int num_free, const int32_t* taken, int block_size, int32_t* taken_out, void* workspace,
                           size_t workspace_bytes, sfa_stream stream) {
  if (rows < 0 || max_blocks_per_seq < 1 || num_blocks < 1 || num_free < 0 || block_size < 1)
    return SFA_ERR_INVALID_ARG;
  if (rows > SFA_PLAN_MAX_REQUESTS || (long long)rows * max_blocks_per_seq >= (1 << 30)) return SFA_ERR_UNSUPPORTED;
  if (!taken || !taken_out || taken == taken_out || !shares || (num_free > 0 && !free_blocks) ||
      (rows > 0 && (!block_table || !held_lens || !keep_lens)))
    return SFA_ERR_INVALID_ARG;
  for (const void* ptr : {(const void*)block_table, (const void*)held_lens, (const void*)keep_lens,
                          (const void*)shares, (const void*)free_blocks, (const void*)taken, (const void*)taken_out,
                          (const void*)workspace})
    if (!aligned(ptr, 4)) return SFA_ERR_INVALID_ARG;
  const size_t need = sfa::blocks_free_workspace_bytes(rows, max_blocks_per_seq);
  if (need && (!workspace || workspace_bytes < need)) return SFA_ERR_WORKSPACE;
  int* status = current_status();
  if (!status) return SFA_ERR_CUDA;
  return done(sfa::launch_blocks_free(block_table, held_lens, keep_lens, rows, max_blocks_per_seq, shares, num_blocks,
                                      free_blocks, num_free, taken, block_size, taken_out, workspace, status,
                                      static_cast<cudaStream_t>(stream)));
}

sfa_status sfa_blocks_compact(const int32_t* block_table, const int32_t* lens, int rows, int max_blocks_per_seq,
                              const int32_t* shares, int num_blocks, const int32_t* free_blocks, int num_free,
                              const int32_t* taken, int block_size, int max_moves, int32_t* table_out,
                              int32_t* shares_out, int32_t* free_out, int32_t* copies, sfa_stream stream) {
  if (rows < 0 || max_blocks_per_seq < 1 || num_blocks < 1 || num_free < 0 || block_size < 1 || max_moves < 0)
    return SFA_ERR_INVALID_ARG;
  if (rows > SFA_PLAN_MAX_REQUESTS || (long long)rows * max_blocks_per_seq >= (1 << 30) ||
      num_blocks > SFA_COMPACT_MAX_BLOCKS)
    return SFA_ERR_UNSUPPORTED;
  if (!taken || !shares || !shares_out || (num_free > 0 && (!free_blocks || !free_out)) ||
      (rows > 0 && (!block_table || !lens || !table_out)) || (max_moves > 0 && !copies) || shares == shares_out ||
      (num_free > 0 && free_blocks == free_out) || (rows > 0 && block_table == table_out))
    return SFA_ERR_INVALID_ARG;
  for (const void* ptr : {(const void*)block_table, (const void*)lens, (const void*)shares, (const void*)free_blocks,
                          (const void*)taken, (const void*)table_out, (const void*)shares_out, (const void*)free_out,
                          (const void*)copies})
    if (!aligned(ptr, 4)) return SFA_ERR_INVALID_ARG;
  int* status = current_status();
  if (!status) return SFA_ERR_CUDA;
  return done(sfa::launch_blocks_compact(block_table, lens, rows, max_blocks_per_seq, shares, num_blocks, free_blocks,
                                         num_free, taken, block_size, max_moves, table_out, shares_out, free_out,
                                         copies, status, static_cast<cudaStream_t>(stream)));
}

static sfa_status copy_blocks(void* kv, float* scales, int group, int row_bytes, int layers, int num_blocks,
                              int block_size, const int32_t* copies, int n, sfa_stream stream) {
  if (layers < 0 || num_blocks < 1 || block_size < 1 || n < 0) return SFA_ERR_INVALID_ARG;
  if (layers == 0 || n == 0) return SFA_OK;
  if (!kv || !copies || !aligned(kv, 16) || !aligned(copies, 4)) return SFA_ERR_INVALID_ARG;
  int* status = current_status();
  if (!status) return SFA_ERR_CUDA;
  return done(sfa::launch_kv_copy_blocks(kv, scales, group, row_bytes, layers, num_blocks, block_size, copies, n,
                                         status, static_cast<cudaStream_t>(stream)));
}

sfa_status sfa_kv_copy_blocks(void* kv, int layers, int num_blocks, int block_size, const int32_t* copies, int n,
                              sfa_stream stream) {
  return copy_blocks(kv, nullptr, 1, SFA_D_QK * 2, layers, num_blocks, block_size, copies, n, stream);
}

sfa_status sfa_kv_copy_blocks_q8(void* kv8, float* scales, int group, int layers, int num_blocks, int block_size,
                                 const int32_t* copies, int n, sfa_stream stream) {
  if (group < 1 || block_size < 1 || block_size % group != 0) return SFA_ERR_INVALID_ARG;
  if (layers > 0 && n > 0 && (!scales || !aligned(scales, 4))) return SFA_ERR_INVALID_ARG;
  return copy_blocks(kv8, scales, group, SFA_D_QK, layers, num_blocks, block_size, copies, n, stream);
}

sfa_status sfa_last_device_status(sfa_stream stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SFA_ERR_CUDA;
  int* status = status_word(dev);
  if (!status) return SFA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return SFA_ERR_CUDA;
  int v = 0;
  if (cudaMemcpy(&v, status, sizeof v, cudaMemcpyDeviceToHost) != cudaSuccess) return SFA_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpy(status, &zero, sizeof zero, cudaMemcpyHostToDevice) != cudaSuccess)
    return SFA_ERR_CUDA;
  return static_cast<sfa_status>(v);
}

}  // extern "C"
