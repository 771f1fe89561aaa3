// sfa_kv_write_q8.cu -- the write of the 8-bit latent cache: each new token's latent row
// (slot_mapping scatter: "RFC: MsModeling 支持 Decode Context Parallel 仿真", 2.1.4.1) is
// stored as e4m3 under a scale shared by a group of `group` consecutive slots.
//
// Scales are powers of two.  The scale of group G becomes
//   s = max(s_before, max over this call's rows of G of 2^ceil(log2(amax / 448)))
// (a call that writes a group's first slot starts it anew: s_before = 0), rows of G that
// the call does not write go from s_before to s, and the new rows are e4m3(x / s).  With
// powers of two the change of scale moves exponents only, so a stored value is rounded
// again only where it becomes subnormal, and a dequantised value is exact in bf16.
//
// Few rows (a decode step) take one launch and a block a group.  More take two: the first takes each
// row's amax and joins it to its group's record in the workspace (atomic max / or / add: the result
// does not depend on their order); the second quantises.  It is launched early (programmatic
// dependent launch) and loads its rows while the first still runs.  The first row of a group to
// arrive there rewrites the group's other rows when its scale rose; the last one stores the scale and
// clears the record, so the workspace is zero between calls.  Groups of one slot need no record and
// take one launch.
//
// Bound: HBM, 1152 bytes read and 576 written a row, and the wait of the second launch for the
// first's atomics: 8885 rows in groups of 16 take 8.9 us (2.3 us of bytes; the first launch 4.0).  Latency for a decode
// step's rows: 64 rows that each join a filled group of 64 take 2.9 to 3.1 us, a chain of slots, rows, the
// group's largest value and, where its scale rose, its other rows.
#include <cuda_fp8.h>
#include <string.h>

#include "sfa_internal.h"

namespace sfa {
namespace {

constexpr int kRowWords = kDQK * 2 / 16;   // 72 x 16 bytes per bf16 row
constexpr int kRow8Words = kDQK / 16;      // 36 x 16 bytes per e4m3 row
constexpr int kThreads = 128, kBlocks = 16;   // a warp a row; 64 warps an SM (32 registers a thread): 8.9 us
                                              // for 8885 rows in groups of 16, 9.4 with the registers free
constexpr int kFewThreads = 512;      // of a block that takes a group, and as many slots a call at most
constexpr int kMinExp = -100, kMaxExp = 120;

struct GroupRecord {
  int need;                    // largest scale exponent of the new rows, - kMinExp + 1
  float old;                   // the group's scale before the call
  int count, done;             // rows of this call; rows quantised
  unsigned long long mask;     // slots of the group that this call writes
  unsigned long long pad;
};
static_assert(sizeof(GroupRecord) == kQ8RecordBytes, "record size");

// |x| of the largest finite value of 8 bf16, as bits
__device__ __forceinline__ unsigned amax_bits(const uint4& x) {
  const unsigned w[4] = {x.x, x.y, x.z, x.w};
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
    if (lo < 0x7f80u) m = max(m, lo);
    if (hi < 0x7f80u) m = max(m, hi);
  }
  return m;
}

// least k with amax <= 448 * 2^k (448 = 1.75 * 2^8), in [kMinExp, kMaxExp]
__device__ __forceinline__ int scale_exp(unsigned bits) {
  const int e = (int)(bits >> 7) - 127;
  const int k = e - 8 + ((bits & 0x7f) > 0x60 ? 1 : 0);
  return bits < 0x80u ? kMinExp : min(max(k, kMinExp), kMaxExp);
}

__device__ __forceinline__ float exp2_int(int k) { return __int_as_float((k + 127) << 23); }

__device__ __forceinline__ unsigned e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// x / s (by its reciprocal where s is a power of two: exact), infinities, which e4m3 does not
// have, to NaN
template <bool kPow2>
__device__ __forceinline__ float scaled(unsigned bf16_bits, float s) {
  const float x = __uint_as_float(bf16_bits << 16);
  return (bf16_bits & 0x7fffu) == 0x7f80u ? __int_as_float(0x7fc00000) : kPow2 ? x * s : x / s;
}

template <bool kPow2>
__device__ __forceinline__ uint2 quantise8(const uint4& x, float s) {
  const unsigned w[4] = {x.x, x.y, x.z, x.w};
  unsigned q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = e4m3x2(scaled<kPow2>(w[i] & 0xffffu, s), scaled<kPow2>(w[i] >> 16, s));
  return make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
}

__device__ __forceinline__ unsigned requantise4(unsigned w, float ratio) {
  unsigned out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    out |= e4m3x2(f.x * ratio, f.y * ratio) << (16 * i);
  }
  return out;
}

// every scale that this file writes is a power of two within [2^-100, 2^120]
__device__ __forceinline__ bool is_pow2(float s) {
  return (__float_as_uint(s) & 0x7fffffu) == 0 && s >= 0x1p-100f;
}

// a warp's row: its words threadIdx.x % 32 + 32 i
struct Row {
  static constexpr int kWords = (kRowWords + 31) / 32;
  uint4 x[kWords];
  long long slot;   // -1: padding, out of range or behind the last row
  int lane;

  __device__ __forceinline__ void load(const int32_t* slots, const uint4* rows, int T, long long num_slots,
                                       int* status) {
    const long long t = (blockIdx.x * (long long)blockDim.x + threadIdx.x) / 32;
    lane = threadIdx.x % 32;
    slot = -1;
    if (t >= T) return;
    slot = slots[t];
    const uint4* src = rows + (size_t)t * kRowWords + lane;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      x[i] = lane + 32 * i < kRowWords ? __ldg(src + 32 * i) : make_uint4(0, 0, 0, 0);
    if (slot >= num_slots) {
      if (status && lane == 0) report_status(status, kStatusBadBlock);
      slot = -1;
    }
  }
  // the row's largest finite magnitude, as bits
  __device__ __forceinline__ unsigned amax() const {
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) m = max(m, amax_bits(x[i]));
    return __reduce_max_sync(0xffffffffu, m);
  }
  __device__ __forceinline__ void store(uint4* kv8, float s) const {
    uint2* dst = reinterpret_cast<uint2*>(kv8 + (size_t)slot * kRow8Words) + lane;
    const bool pow2 = is_pow2(s);
    const float inv = 1.f / s;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      if (lane + 32 * i < kRowWords) dst[32 * i] = pow2 ? quantise8<true>(x[i], inv) : quantise8<false>(x[i], s);
  }
};

// the rows of the group at `base` whose bit of `mask` is clear: from scale `old` to `s`, by the
// threads `thread` of `threads` (out of line: rare, and its words in flight would take the kernels'
// registers)
__device__ __noinline__ void move_group(uint4* base, int group, unsigned long long mask, float old, float s,
                                           int thread, int threads) {
  const float ratio = old / s;
  const int words = group * kRow8Words;
  constexpr int kFly = 6;                      // words in flight a thread
  for (int j0 = thread; j0 < words; j0 += kFly * threads) {
    uint4 w[kFly];
    bool in[kFly];
#pragma unroll
    for (int k = 0; k < kFly; ++k) {
      const int j = j0 + k * threads;
      in[k] = j < words && !((mask >> (j / kRow8Words)) & 1);
      if (in[k]) w[k] = base[j];
    }
#pragma unroll
    for (int k = 0; k < kFly; ++k) {
      if (!in[k]) continue;
      base[j0 + k * threads] = make_uint4(requantise4(w[k].x, ratio), requantise4(w[k].y, ratio),
                                          requantise4(w[k].z, ratio), requantise4(w[k].w, ratio));
    }
  }
}

// the scale that counts as a group's before a call
__device__ __forceinline__ float scale_before(float was, unsigned long long mask) {
  return ((mask & 1) || !(was > 0.f) || was > 3e38f) ? 0.f : was;
}

// Few rows, a block each: the block of a group's first row takes all the group's rows, which it
// finds by reading every slot; the others have nothing to do.
__global__ void __launch_bounds__(kFewThreads) q8_few_kernel(uint4* kv8, float* scales, long long num_slots,
                                                          const int32_t* __restrict__ slots,
                                                          const uint4* __restrict__ rows, int T, int group,
                                                          int* status) {
  constexpr int kKeep = (kQ8MaxWriteGroup * kRowWords + kFewThreads - 1) / kFewThreads;   // words a thread holds
  __shared__ int member_s[kFewThreads], last_s[kQ8MaxWriteGroup], count_s;   // row | offset in the group << 16
  __shared__ unsigned amax_s;
  __shared__ unsigned long long mask_s;
  const int t = blockIdx.x, tid = threadIdx.x;
  uint4 x[kKeep];
  if (tid < kRowWords) x[0] = __ldg(rows + (size_t)t * kRowWords + tid);
  const int mine = __ldg(slots + t), other = tid < T ? __ldg(slots + tid) : -1;
  if (mine < 0) return;
  if (mine >= num_slots) {
    if (tid == 0) report_status(status, kStatusBadBlock);
    return;
  }
  const int g = mine / group, first = g * group, off = other - first;
  const bool in = other >= first && off < group;
  if (tid == 0) {
    count_s = 1;
    amax_s = 0;
    mask_s = 0;
  }
  if (tid < kQ8MaxWriteGroup) last_s[tid] = -1;
  if (__syncthreads_or(in && tid < t)) return;
  const float was = scales[g];
  if (in) {
    member_s[tid == t ? 0 : atomicAdd(&count_s, 1)] = tid | off << 16;
    atomicOr(&mask_s, 1ull << off);
    atomicMax(&last_s[off], tid);              // of rows that name one slot the last is stored
  }
  __syncthreads();
  const int words = count_s * kRowWords;
  const unsigned long long mask = mask_s;
  const auto word = [&](int i) { return rows + (size_t)(member_s[i / kRowWords] & 0xffff) * kRowWords + i % kRowWords; };
  unsigned m = tid < kRowWords ? amax_bits(x[0]) : 0;
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int i = tid + kFewThreads * k;
    if (i >= kRowWords && i < words) x[k] = __ldg(word(i));
  }
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int i = tid + kFewThreads * k;
    if (i >= kRowWords && i < words) m = max(m, amax_bits(x[k]));
  }
  for (int i = tid + kFewThreads * kKeep; i < words; i += kFewThreads) m = max(m, amax_bits(__ldg(word(i))));
  m = __reduce_max_sync(0xffffffffu, m);
  if (tid % 32 == 0) atomicMax(&amax_s, m);
  __syncthreads();
  const float old = scale_before(was, mask), s = fmaxf(old, exp2_int(scale_exp(amax_s)));
  const bool pow2 = is_pow2(s);
  const float inv = 1.f / s;
  uint2* dst = reinterpret_cast<uint2*>(kv8 + (size_t)first * kRow8Words);
  const auto put = [&](int i, const uint4& v) {
    const int member = member_s[i / kRowWords], at = member >> 16;
    if (last_s[at] == (member & 0xffff))
      dst[at * kRowWords + i % kRowWords] = pow2 ? quantise8<true>(v, inv) : quantise8<false>(v, s);
  };
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (tid + kFewThreads * k < words) put(tid + kFewThreads * k, x[k]);
  for (int i = tid + kFewThreads * kKeep; i < words; i += kFewThreads) put(i, __ldg(word(i)));
  if (tid == 0) scales[g] = s;
  if (old > 0.f && s > old) move_group(kv8 + (size_t)first * kRow8Words, group, mask, old, s, tid, kFewThreads);
}

__global__ void __launch_bounds__(kThreads) q8_need_kernel(const float* __restrict__ scales, long long num_slots,
                                                           const int32_t* __restrict__ slots,
                                                           const uint4* __restrict__ rows, int T, int group,
                                                           GroupRecord* rec, int* status) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Row row;
  row.load(slots, rows, T, num_slots, status);
  if (row.slot < 0) return;                      // (the same for all threads of a row)
  const unsigned m = row.amax();
  if (row.lane == 0) {
    const long long g = row.slot / group;
    GroupRecord* r = rec + g;
    atomicMax(&r->need, scale_exp(m) - kMinExp + 1);
    r->old = scales[g];                          // the same value from every row of the group
    atomicAdd(&r->count, 1);
    atomicOr(&r->mask, 1ull << (row.slot - g * group));
  }
}

__global__ void __launch_bounds__(kThreads, kBlocks) q8_store_kernel(uint4* kv8, float* scales, long long num_slots,
                                                            const int32_t* __restrict__ slots,
                                                            const uint4* __restrict__ rows, int T, int group,
                                                            GroupRecord* rec) {
  Row row;
  row.load(slots, rows, T, num_slots, nullptr);
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the records are complete
  if (row.slot < 0) return;
  const long long g = row.slot / group;
  GroupRecord* r = rec + g;
  const unsigned long long mask = __ldcg(&r->mask);
  const float was = __ldcg(&r->old);
  const float old = scale_before(was, mask);
  const float s = fmaxf(old, exp2_int(__ldcg(&r->need) - 1 + kMinExp));
  const int count = __ldcg(&r->count);
  __syncwarp();                                  // every thread has its copy of the record
  int ticket = 0;
  if (row.lane == 0) {
    __threadfence();                             // (its reads come before the count; what is stored below need not)
    ticket = atomicAdd(&r->done, 1);
  }
  row.store(kv8, s);
  if (row.lane == 0 && ticket == count - 1) {    // every row of the group has read the record
    scales[g] = s;
    r->need = 0;
    r->old = 0.f;
    r->count = 0;
    r->done = 0;
    r->mask = 0;
  }
  ticket = __shfl_sync(0xffffffffu, ticket, 0);
  if (ticket == 0 && old > 0.f && s > old)
    move_group(kv8 + (size_t)g * group * kRow8Words, group, mask, old, s, row.lane, 32);
}

// groups of one slot: a row's scale is its own (of a slot named twice parts of both rows are kept, and
// one row's scale)
__global__ void __launch_bounds__(kThreads, kBlocks) q8_row_kernel(uint4* kv8, float* scales, long long num_slots,
                                                          const int32_t* __restrict__ slots,
                                                          const uint4* __restrict__ rows, int T, int* status) {
  Row row;
  row.load(slots, rows, T, num_slots, status);
  if (row.slot < 0) return;
  const float s = exp2_int(scale_exp(row.amax()));
  if (row.lane == 0) scales[row.slot] = s;
  row.store(kv8, s);
}

}  // namespace

cudaError_t launch_kv_write_q8(void* kv8, float* scales, long long num_slots, int group, const int32_t* slots,
                               const void* rows, int T, void* workspace, int* status, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  uint4* kv = static_cast<uint4*>(kv8);
  const uint4* src = static_cast<const uint4*>(rows);
  GroupRecord* rec = static_cast<GroupRecord*>(workspace);
  // One launch for few rows.  A block a group moves the group's other rows when their scale rises, the
  // two launches do it by one warp: rows of as many groups whose scales all rise take 4.2 us at 64 rows
  // and 5.8 at 304 in groups of 64 (two launches 22 and 23), 3.7 and 4.9 in groups of 16 (8.6 and 9.1); a
  // chunk that begins inside a group 6.8 and 8.4 in groups of 64 (13).  Where nothing has to move, as
  // for a prompt from a block's start, the block of a group with many rows is the longer way: 64 to 304
  // rows 8.3-8.4 us in groups of 64 (3.5), 4.3-5.8 in groups of 16 (3.4-3.8); at one row a group 64 rows
  // take 2.9 (4.2), 304 rows 3.8 (4.4), 512 rows 6.4 (4.4).
  if (group > 1 && T <= 2 * device_sm_count() && T <= kFewThreads) {
    q8_few_kernel<<<T, kFewThreads, 0, stream>>>(kv, scales, num_slots, slots, src, T, group, status);
    return cudaGetLastError();
  }
  const unsigned grid = (unsigned)(((long long)T * 32 + kThreads - 1) / kThreads);
  if (group == 1) {
    q8_row_kernel<<<grid, kThreads, 0, stream>>>(kv, scales, num_slots, slots, src, T, status);
    return cudaGetLastError();
  }
  q8_need_kernel<<<grid, kThreads, 0, stream>>>(scales, num_slots, slots, src, T, group, rec, status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, q8_store_kernel, kv, scales, num_slots, slots, src, T, group, rec);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sfa
