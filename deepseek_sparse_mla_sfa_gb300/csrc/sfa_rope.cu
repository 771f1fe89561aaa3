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
// phase, whatever the position; only its top 32 bits go to sincospif.  (A float angle
// would be off by 2^-8 rad at position 131072, a double one costs FP64 instructions, which
// this part issues at 1/64 rate.)
//
// Bound: HBM, each element read and written once.  A thread keeps the phases of its 4 pairs
// and walks rows of the same token, so sines are formed once a token and pair group, not
// once a head.
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
  int interleaved, inverse, in_place;
  float mscale;
  int rows_per_thread;
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

// VP pairs a thread: 4 where every access is aligned for it, else 1
template <typename E, int VP, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  const int groups = p.rot / (2 * VP);                    // pair groups of a row
  const int lanes = kRopeThreads / groups;                // rows side by side in a block
  const int v = threadIdx.x % groups, y = threadIdx.x / groups;
  if (y >= lanes) return;
  const long long rows = (long long)p.T * p.n;
  const long long r0 = (long long)blockIdx.x * lanes * p.rows_per_thread;
  unsigned long long frac[VP];
#pragma unroll
  for (int i = 0; i < VP; ++i) frac[i] = turn_fraction(p.inv_freq[v * VP + i]);
  int have = -1, pos = -1;
  float c[VP], s[VP];
  for (int j = 0; j < p.rows_per_thread; ++j) {
    const long long row = r0 + (long long)j * lanes + y;
    if (row >= rows) return;
    const int t = (int)(row / p.n), hd = (int)(row - (long long)t * p.n);
    if (t != have) {
      have = t;
      pos = p.pos[t];
#pragma unroll
      for (int i = 0; i < VP; ++i) {
        const long long ph = (long long)(frac[i] * (unsigned long long)(long long)pos);
        float sn, cs;
        sincospif((float)(int)(ph >> 32) * 0x1p-31f, &sn, &cs);
        c[i] = cs * p.mscale;
        s[i] = (p.inverse ? -sn : sn) * p.mscale;
      }
    }
    if (pos < 0) continue;                                // a padding row: out stays as it was
    const E* xr = static_cast<const E*>(p.x) + t * p.xt + hd * p.xn;
    E* orow = static_cast<E*>(p.out) + t * p.ot + hd * p.on;
    if constexpr (kInterleaved) {
      alignas(16) E a[2 * VP];
      load_elems<(VP > 1), E, 2 * VP>(xr + 2 * VP * v, a);
#pragma unroll
      for (int i = 0; i < VP; ++i) {
        const float x0 = to_f(a[2 * i]), x1 = to_f(a[2 * i + 1]);
        a[2 * i] = from_f<E>(x0 * c[i] - x1 * s[i]);
        a[2 * i + 1] = from_f<E>(x0 * s[i] + x1 * c[i]);
      }
      store_elems<(VP > 1), E, 2 * VP>(orow + 2 * VP * v, a);
    } else {
      alignas(16) E a[VP];
      alignas(16) E b[VP];
      load_elems<(VP > 1), E, VP>(xr + VP * v, a);
      load_elems<(VP > 1), E, VP>(xr + p.rot / 2 + VP * v, b);
#pragma unroll
      for (int i = 0; i < VP; ++i) {
        const float x0 = to_f(a[i]), x1 = to_f(b[i]);
        a[i] = from_f<E>(x0 * c[i] - x1 * s[i]);
        b[i] = from_f<E>(x0 * s[i] + x1 * c[i]);
      }
      store_elems<(VP > 1), E, VP>(orow + VP * v, a);
      store_elems<(VP > 1), E, VP>(orow + p.rot / 2 + VP * v, b);
    }
    if (!p.in_place)
      for (int d = p.rot + v; d < p.width; d += groups) orow[d] = xr[d];
  }
}

template <typename E, int VP>
cudaError_t launch_typed(RopeParams p, cudaStream_t stream) {
  const int groups = p.rot / (2 * VP), lanes = kRopeThreads / groups;
  const long long rows = (long long)p.T * p.n;
  // rows a thread walks: enough blocks to fill the GPU first, then up to 8 rows of a token
  // behind one set of sines
  const long long fill = 8LL * device_sm_count() * lanes;
  int per = (int)(rows / fill);
  p.rows_per_thread = per < 1 ? 1 : per > 8 ? 8 : per;
  const long long grid = (rows + (long long)lanes * p.rows_per_thread - 1) / ((long long)lanes * p.rows_per_thread);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (p.interleaved)
    rope_kernel<E, VP, true><<<(unsigned)grid, kRopeThreads, 0, stream>>>(p);
  else
    rope_kernel<E, VP, false><<<(unsigned)grid, kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename E>
cudaError_t launch_rope_t(const RopeParams& p, cudaStream_t stream) {
  // 4 pairs a thread need 4 * 2 (interleaved) or 4 (halves) consecutive elements at an
  // address that is a multiple of the access (at most 16 bytes)
  const size_t run = (p.interleaved ? 8 : 4) * sizeof(E), acc = run < 16 ? run : 16;
  const auto ok = [&](const void* q, long long a, long long b) {
    return reinterpret_cast<uintptr_t>(q) % acc == 0 && (a * sizeof(E)) % acc == 0 && (b * sizeof(E)) % acc == 0;
  };
  const bool vec = p.rot % 8 == 0 && ok(p.x, p.xt, p.xn) && ok(p.out, p.ot, p.on) &&
                   (p.interleaved || (p.rot / 2 * sizeof(E)) % acc == 0);
  return vec ? launch_typed<E, 4>(p, stream) : launch_typed<E, 1>(p, stream);
}

}  // namespace

cudaError_t launch_rope(const void* x, long long xt, long long xn, void* out, long long ot, long long on, int dtype,
                        int T, int n, int width, int rot, const int32_t* pos, const double* inv_freq,
                        int interleaved, int inverse, float mscale, cudaStream_t stream) {
  const RopeParams p{x,  out,   pos, inv_freq,    xt,      xn,        ot,     on, T,
                     n,  width, rot, interleaved, inverse, x == out, mscale, 1};
  switch (dtype) {
    case 0: return launch_rope_t<__nv_bfloat16>(p, stream);
    case 1: return launch_rope_t<__half>(p, stream);
    default: return launch_rope_t<float>(p, stream);
  }
}

}  // namespace sfa
