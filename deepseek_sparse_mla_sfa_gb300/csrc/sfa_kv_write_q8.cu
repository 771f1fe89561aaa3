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
// Two launches: the first takes each row's amax and joins it to its group's record in the
// workspace (atomic max / or / add: the result does not depend on their order); the second
// quantises.  It is launched early (programmatic dependent launch) and loads its rows while
// the first still runs.  The first row of a group to arrive there rewrites the group's other
// rows when its scale rose; the last one stores the scale and clears the record, so the
// workspace is zero between calls.  Groups of one slot need no record and take one launch.
//
// Bound: HBM, 1152 bytes read and 576 written a row, and the wait of the second launch for the
// first's atomics: 8885 rows in groups of 16 take 9.5 us (2.3 us of bytes).  Latency for a decode
// step's rows, where four warps take a row (one load each, and a group is rewritten four times as
// fast): 64 rows that each join a filled group of 64 take 3.9 us.
#include <cuda_fp8.h>
#include <string.h>

#include "sfa_internal.h"

namespace sfa {
namespace {

constexpr int kRowWords = kDQK * 2 / 16;   // 72 x 16 bytes per bf16 row
constexpr int kRow8Words = kDQK / 16;      // 36 x 16 bytes per e4m3 row
constexpr int kThreads = 256;         // 8 rows a block, a warp each
constexpr int kFewThreads = 128;      // or one row a block
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

// kRowThreads threads share a row: its words threadIdx.x % kRowThreads + kRowThreads i
template <int kRowThreads>
struct Row {
  static constexpr int kWords = (kRowWords + kRowThreads - 1) / kRowThreads;
  uint4 x[kWords];
  long long slot;   // -1: padding, out of range or behind the last row
  int lane;

  __device__ __forceinline__ void load(const int32_t* slots, const uint4* rows, int T, long long num_slots,
                                       int* status) {
    const long long t = (blockIdx.x * (long long)blockDim.x + threadIdx.x) / kRowThreads;
    lane = threadIdx.x % kRowThreads;
    slot = -1;
    if (t >= T) return;
    slot = slots[t];
    const uint4* src = rows + (size_t)t * kRowWords + lane;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      x[i] = lane + kRowThreads * i < kRowWords ? __ldg(src + kRowThreads * i) : make_uint4(0, 0, 0, 0);
    if (slot >= num_slots) {
      if (status && lane == 0) report_status(status, kStatusBadBlock);
      slot = -1;
    }
  }
  // the row's largest finite magnitude, as bits (every thread of the row calls it; with more
  // than a warp a row, every thread of the block)
  __device__ __forceinline__ unsigned amax() const {
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) m = max(m, amax_bits(x[i]));
    m = __reduce_max_sync(0xffffffffu, m);
    if constexpr (kRowThreads > 32) {
      __shared__ unsigned m_s[kRowThreads / 32];
      if (lane % 32 == 0) m_s[lane / 32] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kRowThreads / 32; ++w) m = max(m, m_s[w]);
    }
    return m;
  }
  __device__ __forceinline__ void store(uint4* kv8, float s) const {
    uint2* dst = reinterpret_cast<uint2*>(kv8 + (size_t)slot * kRow8Words) + lane;
    // every scale that this file writes is a power of two within [2^-100, 2^120]
    const bool pow2 = (__float_as_uint(s) & 0x7fffffu) == 0 && s >= 0x1p-100f;
    const float inv = 1.f / s;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      if (lane + kRowThreads * i < kRowWords)
        dst[kRowThreads * i] = pow2 ? quantise8<true>(x[i], inv) : quantise8<false>(x[i], s);
  }
  // a value of the row's thread 0 to all of them, and a barrier over the row
  __device__ __forceinline__ int broadcast(int v) const {
    if constexpr (kRowThreads > 32) {
      __shared__ int v_s;
      __syncthreads();
      if (lane == 0) v_s = v;
      __syncthreads();
      return v_s;
    } else {
      return __shfl_sync(0xffffffffu, v, 0);
    }
  }
};

template <int kRowThreads>
__global__ void __launch_bounds__(kThreads) q8_need_kernel(const float* __restrict__ scales, long long num_slots,
                                                           const int32_t* __restrict__ slots,
                                                           const uint4* __restrict__ rows, int T, int group,
                                                           GroupRecord* rec, int* status) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Row<kRowThreads> row;
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

template <int kRowThreads>
__global__ void __launch_bounds__(kThreads) q8_store_kernel(uint4* kv8, float* scales, long long num_slots,
                                                            const int32_t* __restrict__ slots,
                                                            const uint4* __restrict__ rows, int T, int group,
                                                            GroupRecord* rec) {
  Row<kRowThreads> row;
  row.load(slots, rows, T, num_slots, nullptr);
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the records are complete
  if (row.slot < 0) return;
  const long long g = row.slot / group;
  GroupRecord* r = rec + g;
  const unsigned long long mask = __ldcg(&r->mask);
  const float was = __ldcg(&r->old);
  const float old = ((mask & 1) || !(was > 0.f) || was > 3e38f) ? 0.f : was;
  const float s = fmaxf(old, exp2_int(__ldcg(&r->need) - 1 + kMinExp));
  const int count = __ldcg(&r->count);
  row.store(kv8, s);
  row.broadcast(0);                              // every thread has its copy of the record
  int ticket = 0;
  if (row.lane == 0) {
    __threadfence();
    ticket = atomicAdd(&r->done, 1);
    if (ticket == count - 1) {                   // every row of the group has read the record
      scales[g] = s;
      r->need = 0;
      r->old = 0.f;
      r->count = 0;
      r->done = 0;
      r->mask = 0;
    }
  }
  ticket = row.broadcast(ticket);
  if (ticket == 0 && old > 0.f && s > old) {
    // the group's rows that this call does not write: from scale `old` to `s`
    const float ratio = old / s;
    uint4* base = kv8 + (size_t)g * group * kRow8Words;
    const int words = group * kRow8Words;
    constexpr int kFly = 6;                      // words in flight a thread
    for (int j0 = row.lane; j0 < words; j0 += kFly * kRowThreads) {
      uint4 w[kFly];
      bool in[kFly];
#pragma unroll
      for (int k = 0; k < kFly; ++k) {
        const int j = j0 + k * kRowThreads;
        in[k] = j < words && !((mask >> (j / kRow8Words)) & 1);
        if (in[k]) w[k] = base[j];
      }
#pragma unroll
      for (int k = 0; k < kFly; ++k) {
        if (!in[k]) continue;
        base[j0 + k * kRowThreads] = make_uint4(requantise4(w[k].x, ratio), requantise4(w[k].y, ratio),
                                                requantise4(w[k].z, ratio), requantise4(w[k].w, ratio));
      }
    }
  }
}

// groups of one slot: a row's scale is its own
template <int kRowThreads>
__global__ void __launch_bounds__(kThreads) q8_row_kernel(uint4* kv8, float* scales, long long num_slots,
                                                          const int32_t* __restrict__ slots,
                                                          const uint4* __restrict__ rows, int T, int* status) {
  Row<kRowThreads> row;
  row.load(slots, rows, T, num_slots, status);
  if (row.slot < 0) return;
  const float s = exp2_int(scale_exp(row.amax()));
  if (row.lane == 0) scales[row.slot] = s;
  row.store(kv8, s);
}

template <int kRowThreads>
cudaError_t launch_rows(uint4* kv8, float* scales, long long num_slots, int group, const int32_t* slots,
                        const uint4* rows, int T, GroupRecord* rec, int* status, cudaStream_t stream) {
  const int threads = kRowThreads > 32 ? kRowThreads : kThreads;
  const unsigned grid = (unsigned)(((long long)T * kRowThreads + threads - 1) / threads);
  if (group == 1) {
    q8_row_kernel<kRowThreads><<<grid, threads, 0, stream>>>(kv8, scales, num_slots, slots, rows, T, status);
    return cudaGetLastError();
  }
  q8_need_kernel<kRowThreads><<<grid, threads, 0, stream>>>(scales, num_slots, slots, rows, T, group, rec, status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, q8_store_kernel<kRowThreads>, kv8, scales, num_slots, slots, rows, T, group, rec);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_write_q8(void* kv8, float* scales, long long num_slots, int group, const int32_t* slots,
                               const void* rows, int T, void* workspace, int* status, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  uint4* kv = static_cast<uint4*>(kv8);
  const uint4* src = static_cast<const uint4*>(rows);
  GroupRecord* rec = static_cast<GroupRecord*>(workspace);
  // four warps a row while that leaves the GPU's blocks few: 64 rows that join filled groups 3.8 us
  // (4.3 with a warp a row), 608 rows 4.2 (4.4), 1216 rows 4.8 (4.3), 2432 rows 8.0 (4.8)
  return T <= 4 * device_sm_count()
             ? launch_rows<kFewThreads>(kv, scales, num_slots, group, slots, src, T, rec, status, stream)
             : launch_rows<32>(kv, scales, num_slots, group, slots, src, T, rec, status, stream);
}

}  // namespace sfa
