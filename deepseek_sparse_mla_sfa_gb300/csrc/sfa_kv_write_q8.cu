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
// quantises.  The first warp of a group to arrive there rewrites the group's other rows
// when its scale rose; the last one stores the scale and clears the record, so the
// workspace is zero between calls.  Groups of one slot need no record and take one launch.
//
// Bound: HBM, 1152 bytes read and 576 written a row; latency for a decode step's rows.
#include <cuda_fp8.h>

#include "sfa_internal.h"

namespace sfa {
namespace {

constexpr int kRowWords = kDQK * 2 / 16;   // 72 x 16 bytes per bf16 row
constexpr int kRow8Words = kDQK / 16;      // 36 x 16 bytes per e4m3 row
constexpr int kThreads = 256;
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

// x / s, infinities (which e4m3 does not have) to NaN
__device__ __forceinline__ float scaled(unsigned bf16_bits, float s) {
  const float x = __uint_as_float(bf16_bits << 16);
  return (bf16_bits & 0x7fffu) == 0x7f80u ? __int_as_float(0x7fc00000) : x / s;
}

__device__ __forceinline__ uint2 quantise8(const uint4& x, float s) {
  const unsigned w[4] = {x.x, x.y, x.z, x.w};
  unsigned q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = e4m3x2(scaled(w[i] & 0xffffu, s), scaled(w[i] >> 16, s));
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

__device__ __forceinline__ unsigned warp_max(unsigned v) { return __reduce_max_sync(0xffffffffu, v); }

// this warp's row into registers; returns its slot, or -1 (padding, out of range)
__device__ __forceinline__ long long load_row(const int32_t* slots, const uint4* rows, int T, long long num_slots,
                                              int t, int lane, uint4 (&x)[3], int* status) {
  if (t >= T) return -1;
  const long long slot = slots[t];
  if (slot < 0) return -1;
  if (slot >= num_slots) {
    if (status && lane == 0) report_status(status, kStatusBadBlock);
    return -1;
  }
  const uint4* src = rows + (size_t)t * kRowWords;
#pragma unroll
  for (int i = 0; i < 3; ++i)
    x[i] = lane + 32 * i < kRowWords ? __ldg(src + lane + 32 * i) : make_uint4(0, 0, 0, 0);
  return slot;
}

__device__ __forceinline__ void store_row(uint4* kv8, long long slot, int lane, const uint4 (&x)[3], float s) {
  uint2* dst = reinterpret_cast<uint2*>(kv8 + (size_t)slot * kRow8Words);
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (lane + 32 * i < kRowWords) dst[lane + 32 * i] = quantise8(x[i], s);
}

__global__ void __launch_bounds__(kThreads) q8_need_kernel(const float* __restrict__ scales, long long num_slots,
                                                           const int32_t* __restrict__ slots,
                                                           const uint4* __restrict__ rows, int T, int group,
                                                           GroupRecord* rec, int* status) {
  const int t = (int)((blockIdx.x * (long long)kThreads + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  uint4 x[3];
  const long long slot = load_row(slots, rows, T, num_slots, t, lane, x, status);
  if (slot < 0) return;
  const unsigned m = warp_max(max(amax_bits(x[0]), max(amax_bits(x[1]), amax_bits(x[2]))));
  if (lane == 0) {
    const long long g = slot / group;
    GroupRecord* r = rec + g;
    atomicMax(&r->need, scale_exp(m) - kMinExp + 1);
    r->old = scales[g];                          // the same value from every row of the group
    atomicAdd(&r->count, 1);
    atomicOr(&r->mask, 1ull << (slot - g * group));
  }
}

__global__ void __launch_bounds__(kThreads) q8_store_kernel(uint4* kv8, float* scales, long long num_slots,
                                                            const int32_t* __restrict__ slots,
                                                            const uint4* __restrict__ rows, int T, int group,
                                                            GroupRecord* rec) {
  const int t = (int)((blockIdx.x * (long long)kThreads + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  uint4 x[3];
  const long long slot = load_row(slots, rows, T, num_slots, t, lane, x, nullptr);
  if (slot < 0) return;
  const long long g = slot / group;
  GroupRecord* r = rec + g;
  const unsigned long long mask = r->mask;
  const float was = r->old;
  const float old = ((mask & 1) || !(was > 0.f) || was > 3e38f) ? 0.f : was;
  const float s = fmaxf(old, exp2_int(r->need - 1 + kMinExp));
  const int count = r->count;
  store_row(kv8, slot, lane, x, s);
  __syncwarp();                                  // every lane has its copy of the record
  int ticket = 0;
  if (lane == 0) {
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
  ticket = __shfl_sync(0xffffffffu, ticket, 0);
  if (ticket == 0 && old > 0.f && s > old) {
    // the group's rows that this call does not write: from scale `old` to `s`
    const float ratio = old / s;
    uint4* base = kv8 + (size_t)g * group * kRow8Words;
    for (int j = lane; j < group * kRow8Words; j += 32) {
      if ((mask >> (j / kRow8Words)) & 1) continue;
      uint4 w = base[j];
      w.x = requantise4(w.x, ratio);
      w.y = requantise4(w.y, ratio);
      w.z = requantise4(w.z, ratio);
      w.w = requantise4(w.w, ratio);
      base[j] = w;
    }
  }
}

// groups of one slot: a row's scale is its own
__global__ void __launch_bounds__(kThreads) q8_row_kernel(uint4* kv8, float* scales, long long num_slots,
                                                          const int32_t* __restrict__ slots,
                                                          const uint4* __restrict__ rows, int T, int* status) {
  const int t = (int)((blockIdx.x * (long long)kThreads + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  uint4 x[3];
  const long long slot = load_row(slots, rows, T, num_slots, t, lane, x, status);
  if (slot < 0) return;
  const unsigned m = warp_max(max(amax_bits(x[0]), max(amax_bits(x[1]), amax_bits(x[2]))));
  const float s = exp2_int(scale_exp(m));
  if (lane == 0) scales[slot] = s;
  store_row(kv8, slot, lane, x, s);
}

}  // namespace

cudaError_t launch_kv_write_q8(void* kv8, float* scales, long long num_slots, int group, const int32_t* slots,
                               const void* rows, int T, void* workspace, int* status, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  const unsigned grid = (unsigned)(((long long)T * 32 + kThreads - 1) / kThreads);
  uint4* kv = static_cast<uint4*>(kv8);
  const uint4* src = static_cast<const uint4*>(rows);
  if (group == 1) {
    q8_row_kernel<<<grid, kThreads, 0, stream>>>(kv, scales, num_slots, slots, src, T, status);
    return cudaGetLastError();
  }
  GroupRecord* rec = static_cast<GroupRecord*>(workspace);
  q8_need_kernel<<<grid, kThreads, 0, stream>>>(scales, num_slots, slots, src, T, group, rec, status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  q8_store_kernel<<<grid, kThreads, 0, stream>>>(kv, scales, num_slots, slots, src, T, group, rec);
  return cudaGetLastError();
}

}  // namespace sfa
