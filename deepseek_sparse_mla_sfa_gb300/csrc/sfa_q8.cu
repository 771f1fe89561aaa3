// sfa_q8.cu -- tcgen05 path of sparse MLA decode over the 8-bit latent cache on sm_103a.
//
// The computation is that of "RFC: MsModeling 支持 Decode Context Parallel 仿真"
// 2.1.4.1-2.1.4.4 and "vllm-ascend PR #18870 解读" 4.3 / 4.5 over rows k_j = c_j e_j (e_j the
// row's e4m3 values, c_j the scale of its group of slots): s_j = scale * c_j * (q . e_j),
// out = sum_j p_j c_j e_j / sum_j p_j, p_j = exp(s_j).
//
// Both contractions run as kind::f8f6f4 on the cache's bytes, with no dequantised copy of
// them; the other operand is split into two e4m3 terms:
//   * q: a bf16 value has 8 significant bits, e4m3 has 4, so q = hi + lo exactly (under a
//     power-of-two scale per head; lo is stored times 16, and only values below 2^-22 of the
//     head's largest are rounded).  hi and lo are two rows of M: 64 heads fill M = 128 and
//     QK^T costs what one bf16 pass over half the bytes would.
//   * weights: P_j = p_j c_j is stored as hi + lo, 8 significant bits as bf16 has, two K
//     steps into the same accumulator.  The reference of the running softmax is the maximum
//     of log2 P_j (so c_j is inside it): P stays in [0, 256], 16 at the maximum that the
//     reference was taken from, where 2^-9 is the spacing of the smallest e4m3 values.
//
// One CTA handles one unit (query token, shard, group of up to 64 heads), whole rows, no
// exchange per tile:
//   * tiles of 96 rows, 3 stages; each row's 576 bytes go to shared memory by 16-byte
//     cp.async into the swizzled operand layout (4 column blocks of 128 bytes, SW128, and
//     the 64 rope bytes, SW64).  An SM's TMA unit needs ~15 ns for a tile::gather4, five of
//     which cover four rows: 1.8 us a tile, more than the matrix instructions take; the
//     copies of four warps are not bound by that unit.
//   * QK^T: S[heads hi|lo, rows] += q[128, 32] E^T, 18 steps, q in TMEM, N = 96;
//   * P.V transposed, O^T[columns, heads] += E^T[128 columns, 32 rows] P^T: four blocks of
//     128 columns, 3 K steps each for hi and lo, N = padded heads.  E^T is the same tile read
//     MN-major.  O takes 4 x 64 columns of TMEM.
// TMEM: q 144 columns, S 96 (two of them for 32 heads or fewer), O^T up to 256.
//
// With few units a cluster of G CTAs shares one: CTA c takes tiles c, c + G, ...; they merge
// (O, m, l) over distributed shared memory at the end.
//
// Warp roles (320 threads): warps 0-3 softmax, O rescale and output (warp w owns TMEM lanes
// 32w..32w+31: 16 heads' hi rows and the same heads' lo rows); warps 4-7 gathers; warp 8
// issues QK^T, warp 9 P.V.  Every wait is bounded; one that gives up records
// SFA_ERR_DEVICE_TIMEOUT and the kernel unwinds without trapping.
#include <atomic>
#include <cuda_fp16.h>
#include <string.h>

#include "sfa_internal.h"
#include "sfa_ptx.cuh"
#include "sfa_resolve.cuh"

namespace sfa {
namespace {

using namespace ptx;

constexpr int kNt = 96;              // selected rows per tile: N of QK^T, K of P.V
constexpr int kStages = 3;
constexpr int kThreads = 320;
constexpr int kWarps = kThreads / 32;
constexpr int kProducerWarp = 4, kProducerWarps = 4, kQkWarp = 8, kPvWarp = 9;
constexpr int kGroupHeads = 64;      // heads of a unit
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kPeak = 4.0f;        // log2 of P at the maximum a reference is taken from
constexpr float kMostP = 8.0f;       // log2 of the largest P before the reference moves

// shared memory map (offsets from a 1024-byte aligned base)
constexpr int kBlk = kNt * 128;                       // 128 latent columns of a tile, SW128
constexpr int kStageBytes = 4 * kBlk + kNt * 64;      // + 64 rope columns, SW64
constexpr int kOffP = kStages * kStageBytes;
constexpr int kPBytes = kGroupHeads * 128;            // P^T [heads x 96 rows] e4m3, K-major SW128 rows
constexpr int kOffList = kOffP + 4 * kPBytes;         // two buffers of hi and lo
constexpr int kListCap = 48 * kNt;                    // resolved rows kept at once (whole tiles)
constexpr int kOffScale = kOffList + kListCap * 4;    // per stage and row: (scale, ceil log2 scale)
constexpr int kOffMisc = kOffScale + kStages * kNt * 8;
// misc: (m, l) per head [64] float2; rescale factors [2][64]; partial maxima [2][4][32]; output
// scales [64]; partial sums [4][32]; flags [16]; TMEM address; per-warp counts
constexpr int kMiscMl = 0, kMiscAlpha = 512, kMiscMax = 1024, kMiscScale = 2048, kMiscSum = 2304,
              kMiscFlags = 2816, kMiscTmem = 2880, kMiscCount = 2896, kMiscBytes = 2944;
constexpr int kOffBar = kOffMisc + kMiscBytes;
constexpr int kBarKvFull = 0, kBarKvEmpty = kBarKvFull + kStages, kBarQReady = kBarKvEmpty + kStages,
              kBarSFull = kBarQReady + 1, kBarSFree = kBarSFull + 2, kBarPReady = kBarSFree + 2,
              kBarPFree = kBarPReady + 2, kBarPvFinal = kBarPFree + 2, kBarMmaFin = kBarPvFinal + 1,
              kBarMmaFin2 = kBarMmaFin + 1, kBarNever = kBarMmaFin2 + 1, kNumBars = kBarNever + 1;
constexpr int kSmemBytes = kOffBar + kNumBars * 8 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(kBlk % 1024 == 0 && kStageBytes % 1024 == 0 && kOffP % 1024 == 0, "operands: 1024-byte alignment");
static_assert(kOffBar % 8 == 0 && kOffScale % 16 == 0, "alignment");
static_assert(2048 * kGroupHeads <= kStages * kStageBytes, "the cluster merge's buffer fits in the stages");
static_assert(kMiscCount + 4 * kWarps <= kMiscBytes, "misc");

constexpr long long kDrainLimit = 1LL << 40;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColQ = 0, kColS = 160, kColO = 256, kColS1 = 400;

struct Q8Params {
  DecodeQ8Params qp;
  int groups;        // head groups of a token
  int group_heads;   // heads of a group (the last may have fewer)
};

// D[tmem] (+)= A * B, e4m3 operands, fp32 accumulation
__device__ __forceinline__ void mma8_ts(uint32_t d, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma8_ss(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
}
// instruction descriptor of kind::f8f6f4: e4m3 A and B (format 0), fp32 D
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// two e4m3 codes of a (low byte) and b
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_h(__half2 v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<uint32_t*>(&v)));
  return r;
}
__device__ __forceinline__ __half2 half2_of(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
  return *reinterpret_cast<__half2*>(&r);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// NH: padded heads of a unit (16, 32 or 64), the N of P.V
template <int NH, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 1) decode_q8_kernel(const Q8Params kp) {
  static_assert(NH == 16 || NH == 32 || NH == 64, "padded head count");
  constexpr int HB = NH / 16;        // blocks of 16 heads; warp w holds block w % HB
  constexpr int R = 4 / HB;          // warps that hold the same heads share a tile's rows
  constexpr int kCols = kNt / R;     // rows of a tile per warp: the hi lanes take the first
  constexpr int kHalf = kCols / 2;   // half of them, the lo lanes the second
  constexpr int kSBufs = NH == 64 ? 1 : 2;
  const DecodeParams& p = kp.qp.p;
  extern __shared__ char smem_raw[];
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  int* list_s = reinterpret_cast<int*>(smem + kOffList);
  float2* rows_s = reinterpret_cast<float2*>(smem + kOffScale);                // [kStages][kNt]
  char* misc = smem + kOffMisc;
  float2* ml_s = reinterpret_cast<float2*>(misc + kMiscMl);
  float* alpha_s = reinterpret_cast<float*>(misc + kMiscAlpha);
  float* max_s = reinterpret_cast<float*>(misc + kMiscMax);
  float* scale_s = reinterpret_cast<float*>(misc + kMiscScale);
  float* lpart_s = reinterpret_cast<float*>(misc + kMiscSum);
  volatile int* flags_s = reinterpret_cast<volatile int*>(misc + kMiscFlags);   // [0] abort, [1] stop, [4 + 4 b + w] rescale
  uint32_t* tmem_base_s = reinterpret_cast<uint32_t*>(misc + kMiscTmem);
  int* wcount_s = reinterpret_cast<int*>(misc + kMiscCount);
  volatile int* abort_s = flags_s;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  uint32_t G;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(G));
  const int unit = blockIdx.x / G;
  const int T = p.B * p.Q;
  // the head groups of a token go out next to each other (they read the same rows), the last
  // shards first (the heaviest of a sparse selection)
  const int hg = unit % kp.groups, tr = unit / kp.groups;
  const int t = tr % T, r = p.n_splits - 1 - tr / T;
  const int h0 = hg * kp.group_heads, nh = min(kp.group_heads, p.h - h0);
  const int b = t / p.Q, qi = t % p.Q;
  const int seq_len = p.seq_lens[b];
  const ShardSel sel = shard_sel(seq_len, seq_len - (p.Q - 1 - qi), r, p.n_splits, p.interleave);
  const int bt_row = p.bt_per_token ? t : b;
  const int32_t* idx = p.topk_idx + (size_t)t * p.top_k;
  const long long wl = p.wait_limit;

  // ---- set-up ----------------------------------------------------------------------
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars[kBarKvFull + s], kProducerWarps);
      mbar_init(&bars[kBarKvEmpty + s], 1);
    }
    mbar_init(&bars[kBarQReady], 4);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars[kBarSFull + x], 1);
      mbar_init(&bars[kBarSFree + x], 4);
      mbar_init(&bars[kBarPReady + x], 4);
      mbar_init(&bars[kBarPFree + x], 1);
    }
    mbar_init(&bars[kBarPvFinal], 1);
    mbar_init(&bars[kBarMmaFin], 1);
    mbar_init(&bars[kBarMmaFin2], 1);
    mbar_init(&bars[kBarNever], 1);         // nothing arrives: the stall test hook waits on it
    for (int x = 0; x < 16; ++x) flags_s[x] = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_base_s, kTmemCols);
    tmem_relinquish();
  }

  // ---- index resolution: count per warp chunk, then ordered compaction into smem ----
  const int chunk = ((p.top_k + kWarps * 32 - 1) / (kWarps * 32)) * 32;
  const int c_begin = min(warp * chunk, p.top_k), c_end = min(c_begin + chunk, p.top_k);
  const bool one_round = chunk <= 8 * 32;
  int row_r[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) row_r[k] = -1;
  {
    int cnt = resolve_chunk<kInterleaved>(p, idx, c_begin, c_end, lane, sel, bt_row, crank == 0 && hg == 0, row_r);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
    if (lane == 0) wcount_s[warp] = cnt;
  }
  __syncthreads();
  int total = 0, off = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int c = wcount_s[w];
    if (w < warp) off += c;
    total += c;
  }
  if (one_round) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const unsigned mask = __ballot_sync(0xffffffffu, row_r[k] >= 0);
      const int o = off + __popc(mask & lanemask_lt());
      if (row_r[k] >= 0 && o < kListCap) list_s[o] = row_r[k];
      off += __popc(mask);
    }
  } else {
    for (int j0 = c_begin; j0 < c_end && off < kListCap; j0 += 32) {
      const int j = j0 + lane;
      const int row = j < c_end ? resolve_row<kInterleaved>(p, bt_row, __ldg(idx + j), sel, false) : -1;
      const unsigned mask = __ballot_sync(0xffffffffu, row >= 0);
      const int o = off + __popc(mask & lanemask_lt());
      if (row >= 0 && o < kListCap) list_s[o] = row;
      off += __popc(mask);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_base_s;
  const int n_tiles = (total + kNt - 1) / kNt;
  const int n_local = n_tiles > (int)crank ? (n_tiles - (int)crank + (int)G - 1) / (int)G : 0;

  auto fail = [&](void) {
    report_status(p.status, kStatusTimeout);
    *abort_s = 1;
  };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, wl));
  };

  // warps 0-3: this lane's head, its reference (log2 units, the same in every warp and lane
  // that holds the head) and this lane's share of its sum
  const int hh = 16 * (warp % HB) + (lane & 15);
  const bool lo_lane = lane >= 16;
  float ref = -INFINITY, l_part = 0.f;
  bool bad_q = false;
  if (warp < 4) {
    // =================== q into TMEM, softmax, O rescale (warps 0-3) ================
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    float c_head;
    {
      const bool have = hh < nh;
      const uint4* qsrc = reinterpret_cast<const uint4*>(p.q + ((size_t)t * p.h + h0 + (have ? hh : 0)) * kDQK);
      uint32_t am = 0;
#pragma unroll 6
      for (int k = 0; k < 36; ++k) {
        const uint4 x = __ldg(qsrc + (lo_lane ? 36 : 0) + k);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) am = max(am, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
      }
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 16));
      bad_q = have && am >= 0x7f80u;            // an infinity or NaN: the head's result is NaN
      const bool zero = !have || bad_q;
      // 2^ke: the least power of two with amax / 2^ke <= 448
      int ke = (int)(am >> 7) - 135 + ((am & 0x7f) > 0x60 ? 1 : 0);
      ke = am < 0x80u || zero ? 0 : max(ke, -100);
      const float down = (p.scale < 0.f ? -1.f : 1.f) * __int_as_float((127 - ke) << 23);
      c_head = fmaxf(fabsf(p.scale) * kLog2e * __int_as_float((127 + ke) << 23), 1e-30f);
#pragma unroll 1
      for (int c = 0; c < 9; ++c) {             // 64 columns of q: 16 columns of TMEM
        uint4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = zero ? make_uint4(0, 0, 0, 0) : __ldg(qsrc + 8 * c + k);
        uint32_t v[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
          uint32_t pr[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = __uint_as_float(w[i] << 16) * down, bb = __uint_as_float(w[i] & 0xffff0000u) * down;
            const uint32_t hi = e4m3x2(a, bb);
            const float2 f = __half22float2(half2_of(hi));
            pr[i] = lo_lane ? e4m3x2((a - f.x) * 16.f, (bb - f.y) * 16.f) : hi;
          }
          v[2 * k] = pr[0] | (pr[1] << 16);
          v[2 * k + 1] = pr[2] | (pr[3] << 16);
        }
        tmem_st16(lane_base + kColQ + 16 * c, v);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarQReady]);
    }
    // S = hi + lo / 16, this lane's term times fa, its partner's times fb
    const float fa = lo_lane ? 0.0625f : 1.f, fb = lo_lane ? 1.f : 0.0625f;
    const int cb = (warp / HB) * kCols + (lo_lane ? kHalf : 0);   // this lane's first tile row
    for (int i = 0; i < n_local; ++i) {
      const int bb = i & 1, sb = kSBufs == 2 ? bb : 0;
      const uint32_t s_par = kSBufs == 2 ? (i >> 1) & 1 : i & 1;
      if (warp == 0) {
        bool go = !*abort_s;
        if (go && !wait_warp(&bars[kBarSFull + sb], s_par)) { fail(); go = false; }
        // P buffer bb is free once P.V of tile i-2 has read it
        if (go && i >= 2 && !wait_warp(&bars[kBarPFree + bb], ((i >> 1) - 1) & 1)) { fail(); go = false; }
        // (the rows' scales were published with the tile, which QK^T waited for)
        if (go && !wait_warp(&bars[kBarKvFull + i % kStages], (i / kStages) & 1)) { fail(); go = false; }
        if (lane == 0) flags_s[1] = go ? 0 : 1;
      }
      named_barrier(1, 128);   // A: the scores of tile i are in TMEM and P buffer bb is free
      if (flags_s[1]) break;
      tc_fence_after();
      uint32_t v[kCols];
      const uint32_t sc_col = lane_base + (sb ? kColS1 : kColS) + (warp / HB) * kCols;
#pragma unroll
      for (int k = 0; k < kCols / 8; ++k) tmem_ld8(sc_col + 8 * k, v + 8 * k);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarSFree + sb]);
      const float2* rs = rows_s + (i % kStages) * kNt + cb;
      const int nvalid = total - kNt * ((int)crank + (int)G * i) - cb;   // of this lane's rows
      float s[kHalf];
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < kHalf; ++j) {
        const float own = __uint_as_float(lo_lane ? v[kHalf + j] : v[j]);
        const float got = __shfl_xor_sync(0xffffffffu, __uint_as_float(lo_lane ? v[j] : v[kHalf + j]), 16);
        const float2 cr = rs[j];
        const float x = fmaf(own, fa, got * fb) * cr.x;
        s[j] = j < nvalid ? x : -INFINITY;
        mx = fmaxf(mx, fmaf(s[j], c_head, cr.y));
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      if (R > 1) {
        float* m4 = max_s + 128 * bb;
        m4[warp * 32 + lane] = mx;
        named_barrier(2, 128);   // B: every warp's maximum of tile i is published
#pragma unroll
        for (int w = 0; w < R; ++w) mx = fmaxf(mx, m4[((warp % HB) + w * HB) * 32 + lane]);
      }
      const float ref_new = (i == 0 || mx > ref + kMostP) ? mx - kPeak : ref;
      const float alpha = i == 0 ? 1.f : ex2(ref - ref_new);
      ref = ref_new;
      uint32_t hi[kHalf / 4], lo[kHalf / 4];
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < kHalf; j += 4) {
        uint32_t h2[2], l2[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float e0 = ex2(fmaf(s[j + 2 * u], c_head, -ref)), e1 = ex2(fmaf(s[j + 2 * u + 1], c_head, -ref));
          sum += e0 + e1;
          // 11 bits are enough under the 8 that hi and lo keep
          const __half2 w = __floats2half2_rn(e0 * rs[j + 2 * u].x, e1 * rs[j + 2 * u + 1].x);
          h2[u] = e4m3x2_h(w);
          l2[u] = e4m3x2_h(__hsub2(w, half2_of(h2[u])));
        }
        hi[j / 4] = h2[0] | (h2[1] << 16);
        lo[j / 4] = l2[0] | (l2[1] << 16);
      }
      l_part = l_part * alpha + sum;
      {
        // this head's row of P^T, bytes cb .. cb + kHalf - 1 of the K-major SW128 row
        char* row = smem + kOffP + bb * 2 * kPBytes + hh * 128;
        constexpr int kW = kHalf % 16 == 0 ? 4 : kHalf % 8 == 0 ? 2 : 1;   // words a store
#pragma unroll
        for (int u = 0; u < kHalf / 4; u += kW) {
          const int byte = cb + 4 * u;
          char* at = row + ((((byte >> 4) ^ (hh & 7)) << 4) | (byte & 15));
          if constexpr (kW == 4) {
            *reinterpret_cast<uint4*>(at) = make_uint4(hi[u], hi[u + 1], hi[u + 2], hi[u + 3]);
            *reinterpret_cast<uint4*>(at + kPBytes) = make_uint4(lo[u], lo[u + 1], lo[u + 2], lo[u + 3]);
          } else if constexpr (kW == 2) {
            *reinterpret_cast<uint2*>(at) = make_uint2(hi[u], hi[u + 1]);
            *reinterpret_cast<uint2*>(at + kPBytes) = make_uint2(lo[u], lo[u + 1]);
          } else {
            *reinterpret_cast<uint32_t*>(at) = hi[u];
            *reinterpret_cast<uint32_t*>(at + kPBytes) = lo[u];
          }
        }
        fence_proxy_async_smem();
      }
      if (warp < HB && !lo_lane) alpha_s[64 * bb + hh] = alpha;
      const bool resc = __any_sync(0xffffffffu, alpha != 1.f);
      if (lane == 0) flags_s[4 + 4 * bb + warp] = resc ? 1 : 0;
      named_barrier(3, 128);   // C: whether O is rescaled, and by what
      if ((flags_s[4 + 4 * bb] | flags_s[5 + 4 * bb] | flags_s[6 + 4 * bb] | flags_s[7 + 4 * bb]) && !*abort_s) {
        // once P.V of the previous tile has completed
        if (!wait_warp(&bars[kBarPFree + (bb ^ 1)], ((i - 1) >> 1) & 1)) fail();
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 4 * HB; ++c) {
          uint32_t o[16];
          tmem_ld16(lane_base + kColO + 16 * c, o);
          tmem_ld_wait();
          const float* al = alpha_s + 64 * bb + 16 * (c % HB);
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al[k]);
          tmem_st16(lane_base + kColO + 16 * c, o);
        }
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarPReady + bb]);
    }
  } else if (warp < kProducerWarp + kProducerWarps) {
    // =================== gathers ===================================================
    // Warp pw copies the tile's rows pw, pw + 4, ...: 24 rows of 36 16-byte words, 27 rounds
    // of 32 lanes.  Up to three tiles are in flight; a tile is signalled when its copies have
    // landed and are visible to the tensor cores' proxy.
    const int pw = warp - kProducerWarp;
    const char* kv = reinterpret_cast<const char*>(p.kv);
    int issued = 0, done = 0, seg = 0;
    bool ok = true;
    float sc[kStages] = {0.f, 0.f, 0.f};
    while (done < n_local && !*abort_s) {
      bool can = issued < n_local && issued - done < kStages;
      if (can && issued >= kStages) {
        const uint32_t par = ((issued / kStages) - 1) & 1;
        can = __all_sync(0xffffffffu, mbar_test(&bars[kBarKvEmpty + issued % kStages], par));
        if (!can && issued == done) {
          if (!(ok = wait_warp(&bars[kBarKvEmpty + issued % kStages], par))) break;
          can = true;
        }
      }
      if (can) {
        const int first = kNt * ((int)crank + (int)G * issued);
        if (first >= (seg + 1) * kListCap) {
          // rare (more valid entries than the list holds): this warp re-resolves the
          // entries of its own rows for the segment that holds this tile
          seg = first / kListCap;
          int ord = 0;
          for (int j0 = 0; j0 < p.top_k; j0 += 32) {
            const int j = j0 + lane;
            const int row = j < p.top_k ? resolve_row<kInterleaved>(p, bt_row, __ldg(idx + j), sel, false) : -1;
            const unsigned mask = __ballot_sync(0xffffffffu, row >= 0);
            const int o = ord + __popc(mask & lanemask_lt()) - seg * kListCap;
            if (row >= 0 && o >= 0 && o < kListCap && o % kProducerWarps == pw) list_s[o] = row;
            ord += __popc(mask);
          }
          __syncwarp();
        }
        const int* rows = list_s + (first - seg * kListCap) + pw;
        const int left = total - first - pw;                 // rows 4 i of this warp with 4 i < left exist
        const uint32_t st = smem_u32(smem + (issued % kStages) * kStageBytes);
#pragma unroll
        for (int i = 0; i < kNt / 4 * 36 / 32; ++i) {
          const int c = 32 * i + lane, rr = c / 36, w = c - 36 * rr;   // word w of row 4 rr + pw
          const bool in = 4 * rr < left;
          const int row = in ? rows[4 * rr] : 0;
          const int y = 4 * rr + pw;
          const uint32_t dst = w < 32 ? st + (w >> 3) * kBlk + y * 128 + (((w & 7) ^ (y & 7)) << 4)
                                      : st + 4 * kBlk + y * 64 + (((w & 3) ^ ((y >> 1) & 3)) << 4);
          cp_async16(dst, kv + (size_t)row * kDQK + 16 * w, in ? 16 : 0);
        }
        cp_commit();
        if (lane < kNt / 4) {
          const float x = 4 * lane < left ? __ldg(kp.qp.scales + (unsigned)rows[4 * lane] / (unsigned)kp.qp.group) : 0.f;
          const int at = issued % kStages;
          if (at == 0) sc[0] = x; else if (at == 1) sc[1] = x; else sc[2] = x;
        }
        ++issued;
        continue;
      }
      // the oldest tile in flight
      switch (issued - done) {
        case 1: cp_wait<0>(); break;
        case 2: cp_wait<1>(); break;
        default: cp_wait<2>(); break;
      }
      const int at = done % kStages;
      if (lane < kNt / 4) {
        const float x = at == 0 ? sc[0] : at == 1 ? sc[1] : sc[2];
        // ceil(log2 x): an upper bound of the weight's exponent, exact for powers of two
        rows_s[at * kNt + 4 * lane + pw] =
            make_float2(x, (float)(((int)__float_as_uint(x) + 0x7fffff) >> 23) - 127.f);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarKvFull + at]);
      ++done;
    }
    if (!ok) fail();
    cp_wait<0>();   // no copy of this CTA may still be landing in shared memory at exit
  } else if (warp == kQkWarp || warp == kPvWarp) {
    // =================== tcgen05 MMA issue: QK^T (warp 8) and P.V (warp 9) ========
    if (lane == 0 && n_local > 0) {
      bool ok = true;
      if (warp == kQkWarp) {
        ok = !p.stall || mbar_wait(&bars[kBarNever], 0, wl);
        ok = ok && mbar_wait(&bars[kBarQReady], 0, wl);
        tc_fence_after();
        const uint32_t id = idesc_e4m3(128, kNt, 0, 0);
        for (int n = 0; ok && n < n_local && !*abort_s; ++n) {
          const int s = n % kStages, sb = kSBufs == 2 ? n & 1 : 0;
          if (!(ok = mbar_wait(&bars[kBarKvFull + s], (n / kStages) & 1, wl))) break;
          // the score buffer is free once the softmax has read the tile before from it
          if (n >= kSBufs &&
              !(ok = mbar_wait(&bars[kBarSFree + sb], (kSBufs == 2 ? (n >> 1) - 1 : n - 1) & 1, wl)))
            break;
          tc_fence_after();
          const uint32_t st = smem_u32(smem + s * kStageBytes);
          const uint32_t d = tmem + (sb ? kColS1 : kColS);
#pragma unroll
          for (int k = 0; k < 16; ++k)
            mma8_ts(d, tmem + kColQ + 8 * k, smem_desc(st + (k >> 2) * kBlk + (k & 3) * 32, 16, 1024, kSwizzle128),
                    id, k > 0);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            mma8_ts(d, tmem + kColQ + 128 + 8 * k, smem_desc(st + 4 * kBlk + k * 32, 16, 512, kSwizzle64), id, 1);
          mma_commit(&bars[kBarSFull + sb]);
        }
      } else {
        // A = E^T: columns 128m..128m+127 of 32 tile rows, MN-major (one SW128 atom wide);
        // B = P^T: NH heads x 32 rows, K-major.  The four blocks' accumulators alternate.
        const uint32_t id = idesc_e4m3(128, NH, 1, 0);
        const uint32_t pt = smem_u32(smem + kOffP);
        for (int n = 0; ok && n < n_local && !*abort_s; ++n) {
          const int s = n % kStages, bb = n & 1;
          if (!(ok = mbar_wait(&bars[kBarPReady + bb], (n >> 1) & 1, wl))) break;
          tc_fence_after();
          const uint32_t st = smem_u32(smem + s * kStageBytes);
#pragma unroll
          for (int k = 0; k < kNt / 32; ++k)
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int m = 0; m < 4; ++m)
                mma8_ss(tmem + kColO + NH * m, smem_desc(st + m * kBlk + 4096 * k, kBlk, 1024, kSwizzle128),
                        smem_desc(pt + (2 * bb + part) * kPBytes + 32 * k, 16, 1024, kSwizzle128), id,
                        (n > 0 || k > 0 || part > 0) ? 1u : 0u);
          mma_commit(&bars[kBarKvEmpty + s]);
          mma_commit(&bars[kBarPFree + bb]);
          if (n == n_local - 1) mma_commit(&bars[kBarPvFinal]);
        }
      }
      if (!ok) fail();
      // every MMA this thread issued has completed before TMEM is released
      uint64_t* fin_bar = &bars[warp == kQkWarp ? kBarMmaFin : kBarMmaFin2];
      mma_commit(fin_bar);
      if (!mbar_wait(fin_bar, 0, kDrainLimit)) report_status(p.status, kStatusTimeout);
    }
  }

  // ---- merge of the cluster's partial results and the output ---------------------
  // Every thread of every CTA of the cluster reaches both cluster barriers.
  __syncwarp();
  bool have_o = false;
  if (warp < 4) {
    if (n_local > 0 && !*abort_s) {
      have_o = wait_warp(&bars[kBarPvFinal], 0);
      if (!have_o) fail();
    }
    // the head's sum: its two lanes of each of its R warps, in a fixed order
    lpart_s[warp * 32 + lane] = l_part;
    named_barrier(2, 128);
    if (warp < HB && !lo_lane) {
      float l = 0.f;
#pragma unroll
      for (int w = 0; w < R; ++w) l += lpart_s[(warp + w * HB) * 32 + lane] + lpart_s[(warp + w * HB) * 32 + lane + 16];
      if (bad_q && have_o) l = __int_as_float(0x7fc00000);
      ml_s[hh] = have_o ? make_float2(ref, l) : make_float2(-INFINITY, 0.f);
    }
  }
  tc_fence_before();
  cluster_sync();   // every CTA's (m, l) is published
  tc_fence_after();
  if (warp < 4 && warp < HB && !lo_lane) {
    // this head's largest reference M, sum L and this CTA's weight 2^(m - M) / L
    float M = -INFINITY;
    for (uint32_t c = 0; c < G; ++c) M = fmaxf(M, ld_cluster_f32(mapa(&ml_s[hh], c)));
    float L = 0.f;
    for (uint32_t c = 0; c < G; ++c) {
      const uint32_t a = mapa(&ml_s[hh], c);
      const float lc = ld_cluster_f32(a + 4u);
      if (lc != 0.f) L += ex2(ld_cluster_f32(a) - M) * lc;
    }
    const float2 mine = ml_s[hh];
    scale_s[hh] = mine.y != 0.f ? ex2(mine.x - M) / L : 0.f;
    if (crank == 0 && hh < nh && !*abort_s)
      p.lse[((size_t)r * T + t) * p.h + h0 + hh] = L != 0.f ? (M + __log2f(L)) * kLn2 : -INFINITY;
  }
  // the merge buffer (in the idle stages): 32-column segment 4m + w, owned by CTA
  // (4m + w) / (16 / G); slot of source CTA c: [lane][NH], 16-byte words swizzled by lane
  float* recv = reinterpret_cast<float*>(smem);
  const int segs = 16 / (int)G;
  const size_t out_at = (((size_t)r * T + t) * p.h + h0) * kDV;
  auto put = [&](int head, int col, float val) {
    if (kp.qp.out_bf16)
      reinterpret_cast<__nv_bfloat16*>(p.out)[out_at + (size_t)head * kDV + col] = __float2bfloat16_rn(val);
    else
      p.out[out_at + (size_t)head * kDV + col] = val;
  };
  __syncwarp();
  if (warp < 4) {
    named_barrier(2, 128);
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
#pragma unroll 1
    for (int c = 0; c < 4 * HB; ++c) {
      const int m = c / HB, hb = 16 * (c % HB);
      uint32_t o[16];
      if (have_o) {
        tmem_ld16(lane_base + kColO + 16 * c, o);
        tmem_ld_wait();
      }
      float f[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) f[k] = have_o ? __uint_as_float(o[k]) * scale_s[hb + k] : 0.f;
      if (G == 1) {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (hb + k < nh && !*abort_s) put(hb + k, 128 * m + 32 * warp + lane, f[k]);
      } else {
        const int seg = 4 * m + warp;
        const uint32_t dst = mapa(recv + ((size_t)(crank * segs + seg % segs) * 32 + lane) * NH, seg / segs);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          st_cluster_v4(dst + 16u * ((hb / 4 + k) ^ (lane & (NH / 4 - 1))), __float_as_uint(f[4 * k]),
                        __float_as_uint(f[4 * k + 1]), __float_as_uint(f[4 * k + 2]), __float_as_uint(f[4 * k + 3]));
      }
    }
  }
  tc_fence_before();
  cluster_sync();   // every CTA's scaled partial O has landed with its owner
  tc_fence_after();
  if (G > 1 && warp < 4 && !*abort_s) {
    for (int sg = warp; sg < segs; sg += 4) {
      const int seg = (int)crank * segs + sg;
#pragma unroll 1
      for (int k4 = 0; k4 < NH / 4; ++k4) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (uint32_t c = 0; c < G; ++c) {
          const float4 x = *reinterpret_cast<const float4*>(
              recv + ((size_t)(c * segs + sg) * 32 + lane) * NH + 4 * (k4 ^ (lane & (NH / 4 - 1))));
          a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
        }
        const float f[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (4 * k4 + k < nh) put(4 * k4 + k, 32 * seg + lane, f[k]);
      }
    }
  }

  // ---- teardown ------------------------------------------------------------------
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

template <int NH, bool kIL>
constexpr auto q8_kernel() {
  return decode_q8_kernel<NH, kIL>;
}

cudaError_t prepare_decode_q8() {
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !attr_set[dev].load(std::memory_order_acquire)) {
    for (auto kernel : {q8_kernel<16, false>(), q8_kernel<16, true>(), q8_kernel<32, false>(), q8_kernel<32, true>(),
                        q8_kernel<64, false>(), q8_kernel<64, true>()}) {
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
      if (e != cudaSuccess) return e;
    }
    attr_set[dev].store(true, std::memory_order_release);
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_decode_q8(const DecodeQ8Params& qp, cudaStream_t stream) {
  const DecodeParams& p = qp.p;
  const long long T = (long long)p.B * p.Q;
  if (T == 0) return cudaSuccess;
  cudaError_t e = prepare_decode_q8();
  if (e != cudaSuccess) return e;
  Q8Params kp;
  kp.qp = qp;
  kp.groups = (p.h + kGroupHeads - 1) / kGroupHeads;
  kp.group_heads = (p.h + kp.groups - 1) / kp.groups;
  const long long units = T * p.n_splits * kp.groups;
  // a unit is shared by up to 8 CTAs while the units fill less than half the GPU and each
  // CTA has a tile of the list
  int G = 1;
  while (G < 8 && units * G * 2 <= device_sm_count() && G * kNt < p.top_k) G *= 2;
  if (units * G > 0x7fffffffLL) return cudaErrorInvalidValue;
  const bool il = p.interleave > 0 && p.n_splits > 1;
  auto kernel = kp.group_heads <= 16   ? (il ? q8_kernel<16, true>() : q8_kernel<16, false>())
                : kp.group_heads <= 32 ? (il ? q8_kernel<32, true>() : q8_kernel<32, false>())
                                       : (il ? q8_kernel<64, true>() : q8_kernel<64, false>());
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3((unsigned)(units * G), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)G;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, kp);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sfa
