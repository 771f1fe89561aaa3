// sfa_rope.cu -- rotary positions of the rope columns that attention reads next to the
// latent ones ("RFC: MsModeling 支持 Decode Context Parallel 仿真", 2.1.4.1: a cache row is
// kv_lora_rank latent + qk_rope_head_dim rotated columns, and so is a query's).
//
// Pair i of row (t, head), angle a = positions[t] * inv_freq[i], scale m:
//   (u, v) = m (x cos a - y sin a, x sin a + y cos a);  inverse: sin -> -sin (the transpose,
//   which is also the gradient of the rotation)
// with (x, y) = columns (2i, 2i+1) (interleaved) or (i, i + rot/2) (halves).
//
// The angle is reduced exactly: inv_freq / 2 pi becomes a 64-bit fraction of a turn by
// integer arithmetic on the double's mantissa, and position * fraction modulo 2^64 is the
// phase, whatever the position; only its top 32 bits go to sincospif.  (The fraction is off by
// 2^-63 of a turn for frequencies below 4 rad a position, so the phase by 2^-32 at the last
// position; by twice as much for each power of two above.)  (A float angle
// would be off by 2^-8 rad at position 131072, a double one costs FP64 instructions, which
// this part issues at 1/64 rate.)
//
// Bound: HBM, each element read and written once.  A block takes some tokens (and, for few
// tokens of many heads, a part of their heads): it forms the cosines and sines of its tokens
// once, in shared memory, and its threads then walk the rows with 8 pairs each (4 of fp32).
// Latency is hidden by eight blocks an SM (32 registers a thread), not by rows in flight a thread:
// 4096 tokens x 64 heads x 64 columns, strided, take 14.9 us; 16.5 us with more registers.  With 4
// pairs a thread and 8 rows each it was 16.4 us, then 20.8 with the registers free, 26 with four
// rows in flight, 33 with eight.  (A kernel that only copies these
// 128-byte pieces between the same strides takes 12.4 to 13.1 us, by 1 to 8 rows in flight a thread.)
#include <cuda_fp16.h>

#include "sfa_internal.h"

namespace sfa {
namespace {

constexpr int kRopeThreads = 256;

struct RopeParams {
  const void* x;
  void* out;
  const int32_t* pos;
  const double* inv_freq;
  long long xt, xn, ot, on;   // row strides in elements
  int T, n, width, rot;
  int interleaved, inverse, in_place, copy_padding;
  float mscale;
  int tokens, heads, head_tiles;   // a block's share; blocks per token group
  uint32_t heads_mul;              // row / heads as (row * heads_mul) >> 32, row < 2^16 (0: heads is 1)
};

template <typename E> __device__ __forceinline__ float to_f(E v);
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename E> __device__ __forceinline__ E from_f(float v);
template <> __device__ __forceinline__ float from_f(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }

// Fraction of a turn per position, in units of 2^-64: f / 2 pi = M 2^(E-1086) C 2^-66 with
// M the 53-bit significand shifted to 64 bits and C = 2^66 / 2 pi.
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
  constexpr unsigned long long kC = 0xA2F9836E4E441529ull;   // floor(2^66 / 2 pi) = floor(2^64 * 2 / pi)
  const unsigned long long u = (unsigned long long)__double_as_longlong(f);
  const int e = (int)((u >> 52) & 0x7ff);
  if (e == 0) return 0;
  const unsigned long long m = ((u & 0xfffffffffffffull) | 0x10000000000000ull) << 11;
  const unsigned long long hi = __umul64hi(m, kC);
  const int sh = e - 1024;
  const unsigned long long s = sh >= 0 ? (sh < 64 ? hi << sh : 0) : (sh > -64 ? hi >> -sh : 0);
  return (u >> 63) ? 0 - s : s;
}

// kVec: p is aligned for the access (16 bytes, or 8 for a run of 8); else one by one
template <bool kVec, typename E, int N>
__device__ __forceinline__ void load_elems(const E* p, E (&v)[N]) {
  constexpr int kBytes = N * (int)sizeof(E);
  if constexpr (kVec && kBytes % 16 == 0) {
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4*>(v)[i] = reinterpret_cast<const uint4*>(p)[i];
  } else if constexpr (kVec && kBytes == 8) {
    *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = p[i];
  }
}
template <bool kVec, typename E, int N>
__device__ __forceinline__ void store_elems(E* p, const E (&v)[N]) {
  constexpr int kBytes = N * (int)sizeof(E);
  if constexpr (kVec && kBytes % 16 == 0) {
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(v)[i];
  } else if constexpr (kVec && kBytes == 8) {
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = v[i];
  }
}

constexpr int kRopeSmem = 32768;   // cosines and sines of a block's tokens
constexpr int kRopeItems = 4;      // most pair groups a thread

// VP pairs a thread: 8 (16-bit types) or 4 where every access is aligned for it, else 1
template <typename E, int VP, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 8) rope_kernel(const RopeParams p) {
  extern __shared__ float2 cs_s[];                        // [tokens][rot / 2], then the positions
  const int pairs = p.rot / 2, groups = pairs / VP;
  int* pos_s = reinterpret_cast<int*>(cs_s + p.tokens * pairs);
  const int t0 = (blockIdx.x / p.head_tiles) * p.tokens, h0 = (blockIdx.x % p.head_tiles) * p.heads;
  const int nt = min(p.tokens, p.T - t0), nh = min(p.heads, p.n - h0);
  for (int x = threadIdx.x; x < nt * pairs; x += kRopeThreads) {
    const int tl = x / pairs, i = x - tl * pairs;
    const int pos = p.pos[t0 + tl];
    const double freq = p.inv_freq[i];
    const unsigned long long frac = turn_fraction(freq);
    const long long ph = (long long)(frac * (unsigned long long)(long long)pos);
    float sn, cs;
    sincospif((float)(int)(ph >> 32) * 0x1p-31f, &sn, &cs);
    if ((__double2hiint(freq) & 0x7ff00000) == 0x7ff00000) sn = cs = __int_as_float(0x7fc00000);   // no angle
    cs_s[x] = make_float2(cs * p.mscale, (p.inverse ? -sn : sn) * p.mscale);
    if (i == 0) pos_s[tl] = pos;
  }
  __syncthreads();
  const int lanes = kRopeThreads / groups;                // rows side by side in a block
  const int v = threadIdx.x % groups, y = threadIdx.x / groups;
  if (y >= lanes) return;
  const E* xb = static_cast<const E*>(p.x) + t0 * p.xt + h0 * p.xn;
  E* ob = static_cast<E*>(p.out) + t0 * p.ot + h0 * p.on;
  const int rows = nt * p.heads;                          // (heads past nh are skipped)
  for (int row = y; row < rows; row += lanes) {
    const int tl = p.heads_mul ? (int)__umulhi((unsigned)row, p.heads_mul) : row, hd = row - tl * p.heads;
    if (hd >= nh || pos_s[tl] < 0) continue;              // a padding row: out stays as it was
    const E* xr = xb + tl * p.xt + hd * p.xn;
    E* orow = ob + tl * p.ot + hd * p.on;
    alignas(16) E a[2 * VP];
    if constexpr (kInterleaved) {
      load_elems<(VP > 1), E, 2 * VP>(xr + 2 * VP * v, a);
    } else {
      load_elems<(VP > 1), E, VP>(xr + VP * v, *reinterpret_cast<E(*)[VP]>(&a[0]));
      load_elems<(VP > 1), E, VP>(xr + pairs + VP * v, *reinterpret_cast<E(*)[VP]>(&a[VP]));
    }
    const float2* cs = cs_s + tl * pairs + VP * v;
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      constexpr int dx = kInterleaved ? 2 : 1, dy = kInterleaved ? 1 : VP;
      const float x0 = to_f(a[dx * i]), x1 = to_f(a[dx * i + dy]);
      const float2 c = cs[i];
      a[dx * i] = from_f<E>(x0 * c.x - x1 * c.y);
      a[dx * i + dy] = from_f<E>(x0 * c.y + x1 * c.x);
    }
    if constexpr (kInterleaved) {
      store_elems<(VP > 1), E, 2 * VP>(orow + 2 * VP * v, a);
    } else {
      store_elems<(VP > 1), E, VP>(orow + VP * v, *reinterpret_cast<E(*)[VP]>(&a[0]));
      store_elems<(VP > 1), E, VP>(orow + pairs + VP * v, *reinterpret_cast<E(*)[VP]>(&a[VP]));
    }
    if (!p.in_place)
      for (int d = p.rot + v; d < p.width; d += groups) orow[d] = xr[d];
  }
  if (p.copy_padding && !p.in_place)                      // or is x's
    for (int tl = 0; tl < nt; ++tl)
      for (int hd = y; hd < nh && pos_s[tl] < 0; hd += lanes)
        for (int d = v; d < p.width; d += groups) ob[tl * p.ot + hd * p.on + d] = xb[tl * p.xt + hd * p.xn + d];
}

template <typename E, int VP>
cudaError_t launch_typed(RopeParams p, cudaStream_t stream) {
  const int pairs = p.rot / 2, groups = pairs / VP, lanes = kRopeThreads / groups;
  // rows a block takes: enough blocks to fill the GPU 4 times over first, then up to
  // kRopeItems rows a thread; whole tokens, as many as the cosines have room for, or a part
  // of one token's heads
  const long long want = (long long)p.T * p.n / (4LL * device_sm_count());
  const long long most = (long long)lanes * kRopeItems;
  const long long rows = want < lanes ? lanes : want > most ? most : want;
  p.tokens = (int)(rows / p.n);
  const int room = kRopeSmem / (pairs * 8 + 4);
  p.tokens = p.tokens < 1 ? 1 : p.tokens > room ? room : p.tokens;
  p.tokens = p.tokens < p.T ? p.tokens : p.T;
  p.heads = (long long)p.n <= rows ? p.n : (int)rows;
  p.head_tiles = (p.n + p.heads - 1) / p.heads;
  p.heads = (p.n + p.head_tiles - 1) / p.head_tiles;
  if ((long long)p.tokens * p.heads >= 65536) return cudaErrorInvalidValue;
  p.heads_mul = p.heads == 1 ? 0 : 0xffffffffu / (unsigned)p.heads + 1;
  const long long grid = (long long)((p.T + p.tokens - 1) / p.tokens) * p.head_tiles;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  const size_t smem = (size_t)p.tokens * (pairs * 8 + 4);
  if (p.interleaved)
    rope_kernel<E, VP, true><<<(unsigned)grid, kRopeThreads, smem, stream>>>(p);
  else
    rope_kernel<E, VP, false><<<(unsigned)grid, kRopeThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename E>
cudaError_t launch_rope_t(const RopeParams& p, cudaStream_t stream) {
  // VP pairs a thread need 2 VP (interleaved) or VP (halves) consecutive elements at an address that
  // is a multiple of the access (at most 16 bytes)
  const auto fits = [&](int vp) {
    const size_t run = (p.interleaved ? 2 : 1) * vp * sizeof(E), acc = run < 16 ? run : 16;
    const auto ok = [&](const void* q, long long a, long long b) {
      return reinterpret_cast<uintptr_t>(q) % acc == 0 && (a * sizeof(E)) % acc == 0 && (b * sizeof(E)) % acc == 0;
    };
    return p.rot % (2 * vp) == 0 && ok(p.x, p.xt, p.xn) && ok(p.out, p.ot, p.on) &&
           (p.interleaved || (p.rot / 2 * sizeof(E)) % acc == 0);
  };
  // 8 pairs of a 16-bit type are 16-byte accesses: 4096 x 64 x 64 columns 14.9 us, by 4 pairs 16.4
  if (sizeof(E) == 2 && fits(8)) return launch_typed<E, sizeof(E) == 2 ? 8 : 4>(p, stream);
  return fits(4) ? launch_typed<E, 4>(p, stream) : launch_typed<E, 1>(p, stream);
}

}  // namespace

cudaError_t launch_rope(const void* x, long long xt, long long xn, void* out, long long ot, long long on, int dtype,
                        int T, int n, int width, int rot, const int32_t* pos, const double* inv_freq,
                        int interleaved, int inverse, int copy_padding, float mscale, cudaStream_t stream) {
  const RopeParams p{x,  out,   pos, inv_freq,    xt,      xn,        ot,     on, T,
                     n,  width, rot, interleaved, inverse, x == out, copy_padding, mscale, 1, 1, 1, 0};
  switch (dtype) {
    case 0: return launch_rope_t<__nv_bfloat16>(p, stream);
    case 1: return launch_rope_t<__half>(p, stream);
    default: return launch_rope_t<float>(p, stream);
  }
}

}  // namespace sfa
