// sfa_q8.cu -- tcgen05 path of sparse MLA decode over the 8-bit latent cache on sm_103a.
//
// The computation is that of "RFC: MsModeling 支持 Decode Context Parallel 仿真"
// 2.1.4.1-2.1.4.4 and "vllm-ascend PR #18870 解读" 4.3 / 4.5 over rows k_j = c_j e_j (e_j the
// row's e4m3 values, c_j the scale of its group of slots): s_j = scale * c_j * (q . e_j),
// out = sum_j p_j c_j e_j / sum_j p_j, p_j = exp(s_j).
//
// Both contractions run as 8-bit products (kind::f8f6f4, kind::mxf8f6f4) on the cache's bytes, with
// no dequantised copy of them; the other operand is split into two e4m3 terms:
//   * q: a bf16 value has 8 significant bits, e4m3 has 4, so q = hi + lo exactly (under a
//     power-of-two scale per head; lo is stored times 16, and only values below 2^-22 of the
//     head's largest are rounded).  hi and lo are two rows of M: 64 heads fill M = 128 and
//     QK^T costs what one bf16 pass over half the bytes would.
//   * weights: P_j = p_j c_j is stored as hi + lo / 16, 8 significant bits as bf16 has, two K steps
//     into the same accumulator, under a power-of-two scale for each head and 32 rows
//     (kind::mxf8f6f4).  The largest of the 32 lies in (2^7, 2^8], so a weight is off by 2^-9 of itself,
//     or by 2^-21 of that largest one where this is more (half of 2^-9, the spacing of e4m3's smallest
//     values, by lo's 2^-4).  Under one scale for the whole list a row that takes most of a head's weight
//     left those below 2^-13 of it no value at all: out was off by up to 0.9 of itself.
//     The scales count from a reference that O of a head has; it is the first tile's largest, and
//     moves only where a block is 2^24 above it.  The sum of the weights is fp32 and has a reference
//     of its own, the largest so far.  out is divided by the sum of the weights as they are stored (large
//     ones rounded, small ones not), so that a row with most of the weight is not off by the rounding
//     of its own: error of the shapes below 2.3e-4 to 2.9e-4 of out, divided by lse's sum 6.6e-4 to 7.2e-4.
//
// One CTA handles one unit (query token, shard, group of up to 64 heads), whole rows, no
// exchange per tile:
//   * tiles of 96 rows, 3 stages, in the swizzled operand layout: 4 column blocks of 128
//     latent bytes a row (SW128) and the 64 rope bytes (SW64), all by TMA tile::gather4 from the
//     elected lanes of four warps;
//   * QK^T: S[heads hi|lo, rows] += q[128, 32] E^T, 18 steps, q in TMEM, N = 96;
//   * P.V transposed, O^T[columns, heads] += E^T[128 columns, 32 rows] P^T: four blocks of
//     128 columns, 3 K steps, each hi and then lo with the same A, which the second takes from
//     the collector buffer (at N = 64 the read of A from shared memory, 4 KB, takes longer than
//     the products: 48.9 -> 47.4 us below).  E^T is the same tile read MN-major.
// TMEM: q 144 columns, scales 12, S 96 (two of them for 32 heads or fewer), O^T up to 256.
//
// With few units a cluster of G CTAs shares one: CTA c takes every G-th 96 entries of the list; they merge
// (O, m, l) over distributed shared memory at the end.
//
// Warp roles (640 threads): warps 0-7 softmax (each 8 heads whole); 8 issues QK^T, 9 P.V; 10-13
// the gathers; 14 the rows' scales and the later segments of a long list; 16-19 bring the weights'
// scales to TMEM and scale O where a reference moved; all take a part in the output.  At the start
// warps 0-7 and 16-19 bring q to TMEM while 8-15 resolve the list.  Every wait is bounded; one that gives up records
// SFA_ERR_DEVICE_TIMEOUT and the kernel unwinds without trapping.
//
// Measured (device time in a graph): 64 tokens x 128 heads x 2048 rows 45.4 us, 256 tokens x 64
// heads x 2048 rows 89.9 us (their bytes alone: 13.9 and 50.4 us), 32 tokens x 16 heads x 8192
// rows in four shards 47.4 us (22.7).  Without the second sum 44.6, 88.5, 46.7; with one scale for
// the whole list, and O's reference moving with the largest weight, 45.2, 89.8, 47.0.  Bound: at 64
// heads a tile's MMAs take most of its time and the rest is the chain scores -> softmax -> P.V with
// one score buffer (TMEM is full); the first scores come after 12,600-14,600 cycles (launch, list,
// table, q and the first rows follow one another), the end takes 5,000, and a second round of
// units a whole one's time.
// Taken back: 64-row tiles in 4 or 5 stages (63 vs 61 us at the time), part of the columns by
// cp.async (64-94 vs 61), rows prefetched to L2 (67 vs 61, 72 vs 49), P.V handed over in
// three parts (51.5 vs 49.0), references moved two groups of heads at a time (47.5 vs 45.9).
#include <atomic>
#include <cuda.h>
#include <cuda_fp16.h>
#include <mutex>
#include <string.h>

#include "sfa_internal.h"
#include "sfa_ptx.cuh"
#include "sfa_resolve.cuh"

namespace sfa {
namespace {

using namespace ptx;

constexpr int kNt = 96;              // selected rows per tile: N of QK^T, K of P.V
constexpr int kStages = 3;
constexpr int kThreads = 640;
constexpr int kSoftWarps = 8, kQWarps = 12;
constexpr int kListWarps = 8, kQkWarp = 8, kPvWarp = 9, kProducerWarp = 10, kProducerWarps = 4, kRowWarp = 14,
              kFixWarp = 16, kFixWarps = 4;
constexpr int kGroupHeads = 64;      // heads of a unit
constexpr int kQParts = (kGroupHeads + kQWarps - 1) / kQWarps;   // copies of q, kQWarps heads each
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kWBlock = 32;          // weights under one scale: K of an MMA
constexpr float kPeak = 8.0f;        // log2 of the most that a block's largest weight is stored as (e4m3 ends at 448)
constexpr float kFine = 0x1p-6f;     // weights from here on are stored to 2^-9 of themselves
constexpr float kRise = 24.0f;       // log2 of what a block's scale may rise above its head's reference
constexpr float kFall = 120.0f;      // and fall below it (a scale is 2^-127 at least)

// shared memory map (offsets from a 1024-byte aligned base)
constexpr int kBlk = kNt * 128;                       // 128 latent columns of a tile, SW128
constexpr int kStageBytes = 4 * kBlk + kNt * 64;      // + 64 rope columns, SW64
constexpr int kOffP = kStages * kStageBytes;
constexpr int kPBytes = kGroupHeads * 128;            // P^T [heads x 96 rows] e4m3, K-major SW128 rows
constexpr int kOffList = kOffP + 4 * kPBytes;         // two buffers of hi and lo
constexpr int kListCap = 64 * kNt;                    // resolved rows kept at once (whole tiles)
constexpr int kOffScale = kOffList + kListCap * 4;    // per stage and two rows: scales, then their log2
constexpr int kOffInv = kOffScale + kStages * kNt * 8;  // 1 / scale
constexpr int kOffMisc = kOffInv + kStages * kNt * 4;
constexpr int kMiscMl = 0, kMiscAlpha = 512, kMiscScale = 1024, kMiscC = 1280, kMiscFlags = 1536, kMiscTmem = 1540,
              kMiscMoved = 1544, kMiscCount = 1560, kMiscSeg = 1600, kMiscSf = 1616, kMiscRef = 2128, kMiscKept = 2384, kMiscBytes = 2640;
constexpr int kOffBar = kOffMisc + kMiscBytes;
constexpr int kBarKvFull = 0, kBarKvEmpty = kBarKvFull + kStages, kBarRows = kBarKvEmpty + kStages,
              kBarSegFree = kBarRows + kStages, kBarSegFull = kBarSegFree + 1, kBarQLoad = kBarSegFull + 1, kBarQReady = kBarQLoad + kQParts,
              kBarSFull = kBarQReady + 1, kBarSFree = kBarSFull + 2, kBarAReady = kBarSFree + 2, kBarPReady = kBarAReady + 2,
              kBarPFree = kBarPReady + 2, kBarPvFinal = kBarPFree + 2, kBarMmaFin = kBarPvFinal + 1,
              kBarMmaFin2 = kBarMmaFin + 1, kBarNever = kBarMmaFin2 + 1, kNumBars = kBarNever + 1;
constexpr int kSmemBytes = kOffBar + kNumBars * 8 + 1024;
static_assert(kNt % (4 * kProducerWarps) == 0, "whole row groups a producer");
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(kBlk % 1024 == 0 && kStageBytes % 1024 == 0 && kOffP % 1024 == 0, "operands: 1024-byte alignment");
static_assert(kOffBar % 8 == 0 && kOffScale % 16 == 0, "alignment");
static_assert(2048 * kGroupHeads <= kStages * kStageBytes, "the cluster merge fits in the stages");
// q on its way to TMEM, in stages 1 and 2: 64 rows of 576 bf16, then in place 576 hi and 576 lo bytes
constexpr int kQPitch = 2 * kDQK;
constexpr int kOffTmp = kStageBytes + kGroupHeads * kQPitch;   // behind it: the resolved list before its compaction
constexpr int kTmpCap = (kStages * kStageBytes - kOffTmp) / 4;
static_assert(kTmpCap >= 8192, "q and a list of 8192 entries fit in stages 1 and 2");
static_assert(kMiscCount + 4 * (kListWarps + 1) <= kMiscSeg, "misc");


// A wait that is not over at once goes on outside of the kernel's own code, which every launch
// fetches anew: with the loops in line 64 tokens x 128 heads x 2048 rows take 45.7 us, without 45.0
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, long long limit, uint64_t cap_ns) {
  return mbar_wait(bar, parity, limit, cap_ns);
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, long long limit, uint64_t cap_ns = 4000000000ull) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, limit, cap_ns);
}
constexpr long long kDrainLimit = 1LL << 40;
constexpr uint64_t kLanded = 100000000ull;   // ns: copies in flight have landed long before (a tile that was given up
                                             // half issued never completes its barrier)
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColQ = 0, kColS = 160, kColO = 256, kColS1 = 400;   // S1 for up to 32 heads
// scales of P.V's operands: of E^T all 1; of two buffers of P^T, two words (64 heads) for hi and two for lo
constexpr uint32_t kColSfE = 144, kColSfP = 148;

// 16-byte word w of a converted row of q: moved so that eight rows' are in different banks
__device__ __forceinline__ int q_word(int row, int w) { return w ^ (w < 32 ? row & 7 : row & 3); }

struct Q8Params {
  DecodeQ8Params qp;
  int groups;        // head groups of a token
  int group_heads;   // heads of a group (the last may have fewer)
  int num_rows;      // rows of the cache: the index that the gathers read as zeros
  uint32_t bs_mul, bs_shift, gr_mul, gr_shift;   // division by block_size and by group
  uint32_t T_mul, T_shift, Q_mul, Q_shift;       // by the tokens and by the tokens of a sequence
};

// n / d for 0 <= n < 2^31 as (n * mul) >> shift, mul = ceil(2^shift / d), shift = 31 + ceil(log2 d)
// (mul < 2^32, and the error n (mul d - 2^shift) / (d 2^shift) stays below 1 / d)
__device__ __forceinline__ int div_by(int n, uint32_t mul, uint32_t shift) {
  return (int)(((uint64_t)(uint32_t)n * mul) >> shift);
}
void divisor(int d, uint32_t& mul, uint32_t& shift) {
  shift = 31;
  while ((1ull << (shift - 31)) < (uint64_t)d) ++shift;
  mul = (uint32_t)(((1ull << shift) + (uint64_t)d - 1) / (uint64_t)d);
}

// D[tmem] (+)= A * B, e4m3 operands, fp32 accumulation.  A shared-memory descriptor's high
// word (strides, swizzle) is a constant of the operand; the low word is the address.
template <uint32_t kHi>
__device__ __forceinline__ void mma8_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kHi)
      : "memory");
}
// The same with a scale for each row of A and of B, 32 of K: ue8m0 bytes in TMEM, a row's at lane row %
// 32 (of all four quadrants) of word row / 32, the byte that `idesc` names.
// (kFirst: A stays in the collector buffer, and the next MMA, with the same A, takes it from
// there instead of from shared memory)
template <uint32_t kHiA, uint32_t kHiB, bool kFirst>
__device__ __forceinline__ void mma8_scaled_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t sf_a,
                                               uint32_t sf_b, uint32_t acc) {
  if constexpr (kFirst)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %7};\n\tmov.b64 db, {%2, %8};\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X.collector::a::fill [%0], da, db, %3, [%5], "
        "[%6], p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "r"(sf_a), "r"(sf_b), "n"(kHiA), "n"(kHiB)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %7};\n\tmov.b64 db, {%2, %8};\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X.collector::a::lastuse [%0], da, db, %3, "
        "[%5], [%6], p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "r"(sf_a), "r"(sf_b), "n"(kHiA), "n"(kHiB)
        : "memory");
}
// the words of a shared-memory matrix descriptor (addresses and strides in 16-byte units)
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return (saddr >> 4) | ((lbo >> 4) << 16);
}
constexpr uint32_t desc_hi(uint32_t sbo, uint32_t swizzle) { return (sbo >> 4) | (1u << 14) | (swizzle << 29); }
// one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// instruction descriptor of kind::f8f6f4: e4m3 A and B (format 0), fp32 D
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// of kind::mxf8f6f4 with block scales: the same, ue8m0 scales, A's byte 0 and B's byte `sf_b`
__host__ __device__ constexpr uint32_t idesc_e4m3_scaled(int M, int N, int a_mn, int b_mn, int sf_b) {
  return (idesc_e4m3(M, N, a_mn, b_mn) & ~(1u << 4)) | (static_cast<uint32_t>(sf_b) << 4) | (1u << 23);
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// 16 lanes x 16 columns: thread i gets lane i / 4, columns 2 (i % 4) and + 1, in r[0..1], lane
// i / 4 + 8, the same columns, in r[2..3]; columns 8 .. 15 in r[4..7]
__device__ __forceinline__ void tmem_ld_16x16(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// two e4m3 codes, v.x's in the low byte, and back
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

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A CTA's part of the selected list: of the G CTAs that share a unit, CTA c takes the blocks of 96
// entries c, c + G, ... (each resolves its own entries only: with every CTA resolving the whole list
// one token x 16 heads x 16384 rows took 72 us, not 34)
struct ListPart {
  const int32_t* idx;
  int top_k, g_shift, crank;
  __device__ __forceinline__ int entries() const {
    const int blocks = (top_k + kNt - 1) / kNt, g = 1 << g_shift;
    if (blocks <= crank) return 0;
    const int mine = ((blocks - crank + g - 1) >> g_shift) * kNt;
    return ((blocks - 1) & (g - 1)) == crank ? mine - (blocks * kNt - top_k) : mine;
  }
  // where entry x of the part is in the list
  __device__ __forceinline__ int at(int x) const {
    return x + kNt * (x / kNt * ((1 << g_shift) - 1) + crank);
  }
};

// entries j0 + 32 k + lane < end (k < 8) of the part, -1 behind its end
__device__ __forceinline__ void load8(const ListPart& list, int j0, int end, int lane, int (&pos)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int x = j0 + 32 * k + lane;
    pos[k] = x < end ? __ldg(list.idx + list.at(x)) : -1;
  }
}
// their rows, -1 for those that do not resolve to a row of this unit; returns how many do
template <bool kInterleaved>
__device__ __forceinline__ int resolve8(const Q8Params& kp, int (&pos)[8], const ShardSel& sel, int bt_row, bool report,
                                        int (&row)[8]) {
  const DecodeParams& p = kp.qp.p;
  const int32_t* table = p.block_table + (size_t)bt_row * p.max_blocks;
  int cnt = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const bool in = sel.has_fixed<kInterleaved>(pos[k]);
    const int blk = in ? div_by(pos[k], kp.bs_mul, kp.bs_shift) : 0;
    pos[k] = in ? pos[k] - blk * p.block_size : -1;      // the offset in its block
    row[k] = in && blk < p.max_blocks ? __ldg(table + blk) : -1;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const bool valid = row[k] >= 0 && row[k] < p.num_blocks;
    if (pos[k] >= 0 && !valid && report) report_status(p.status, kStatusBadBlock);
    cnt += valid;
    row[k] = valid ? row[k] * p.block_size + pos[k] : -1;
  }
  return cnt;
}

// two fp32 in a register pair
__device__ __forceinline__ uint64_t pack2u(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) { return pack2u(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

__device__ __noinline__ void give_up(int* status, volatile int* abort_s) {
  report_status(status, kStatusTimeout);
  *abort_s = 1;
}
// NH: padded heads of a unit (32 or 64), the N of P.V
template <int NH, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 1)
    decode_q8_kernel(const __grid_constant__ CUtensorMap tmap_lat, const __grid_constant__ CUtensorMap tmap_rope,
                     const __grid_constant__ Q8Params kp) {
  static_assert(NH == 32 || NH == 64, "padded head count");
  constexpr int HB = NH / 16;             // blocks of 16 heads: TMEM lanes 32x.. hold block x < HB
  constexpr int kSBufs = NH == 64 ? 1 : 2;
  const DecodeParams& p = kp.qp.p;
  extern __shared__ char smem_raw[];
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  int* list_s = reinterpret_cast<int*>(smem + kOffList);
  float4* rows_s = reinterpret_cast<float4*>(smem + kOffScale);          // [kStages][kNt / 2]
  float* inv_s = reinterpret_cast<float*>(smem + kOffInv);               // [kStages][kNt]
  char* misc = smem + kOffMisc;
  float2* ml_s = reinterpret_cast<float2*>(misc + kMiscMl);              // [64] (m, l)
  float* alpha_s = reinterpret_cast<float*>(misc + kMiscAlpha);          // [2][64] rescale factors
  uint8_t* moved_s = reinterpret_cast<uint8_t*>(misc + kMiscMoved);      // [2][8] whether 8 heads' references moved
  uint32_t* sf_s = reinterpret_cast<uint32_t*>(misc + kMiscSf);          // [2][64] the scales of hi's three blocks, as ue8m0
  float* below_s = reinterpret_cast<float*>(misc + kMiscRef);            // [64] O's reference, relative to that of (m, l)
  float* kept_s = reinterpret_cast<float*>(misc + kMiscKept);            // [64] l of the weights as they are stored
  float* scale_s = reinterpret_cast<float*>(misc + kMiscScale);          // [64] output scales
  float* qc_s = reinterpret_cast<float*>(misc + kMiscC);                 // [64] score scale, NaN for a bad head
  volatile int* abort_s = reinterpret_cast<volatile int*>(misc + kMiscFlags);
  uint32_t* tmem_base_s = reinterpret_cast<uint32_t*>(misc + kMiscTmem);
  int* seg_s = reinterpret_cast<int*>(misc + kMiscSeg);                  // where the next list segment starts: entry, ordinal
  int* wcount_s = reinterpret_cast<int*>(misc + kMiscCount);             // [kListWarps + 1]: counts, total

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  uint32_t G;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(G));
  const int g_shift = 31 - __clz((int)G);
  const int unit = (int)(blockIdx.x >> g_shift);
  const int T = p.B * p.Q;
  // the head groups (1 or 2) of a token go out next to each other (they read the same rows),
  // the last shards first (the heaviest of a sparse selection)
  const int hg = unit & (kp.groups - 1), tr = unit >> (kp.groups - 1);
  const int ts = div_by(tr, kp.T_mul, kp.T_shift), t = tr - ts * T, r = p.n_splits - 1 - ts;
  const int h0 = hg * kp.group_heads, nh = min(kp.group_heads, p.h - h0);
  const int b = div_by(t, kp.Q_mul, kp.Q_shift), qi = t - b * p.Q;
  const int bt_row = p.bt_per_token ? t : b;
  const ListPart list{p.topk_idx + (size_t)t * p.top_k, p.top_k, g_shift, (int)crank};
  const int entries = list.entries();
  const uint4* qsrc = reinterpret_cast<const uint4*>(p.q + ((size_t)t * p.h + h0) * kDQK);
  const long long wl = p.wait_limit;

  // ---- set-up ----------------------------------------------------------------------
  // Warps 0-7 and 16-19 bring q into TMEM; meanwhile warps 8-15 resolve the list and start the
  // gathers.  The first loads of both go out before anything waits.
  const int wq = warp < kSoftWarps ? warp : warp - kListWarps;    // of the kQWarps that bring q
  const int chunk = ((entries + kListWarps * 32 - 1) / (kListWarps * 32)) * 32;
  const int c_begin = min((warp - kSoftWarps) * chunk, entries), c_end = min(c_begin + chunk, entries);
  int pos_r[8];
  // (a list of one round, 8 entries a lane, is loaded to registers, a longer one to shared
  // memory, where each warp then compacts its part in place; the longest come round by round)
  const bool one_round = chunk <= 256, staged = !one_round && kListWarps * chunk <= kTmpCap;
  int* const tmp = reinterpret_cast<int*>(smem + kOffTmp) + (warp - kSoftWarps) * chunk;
  if (warp >= kSoftWarps && warp < kFixWarp) {
    if (one_round) load8(list, c_begin, c_end, lane, pos_r);
    if (staged)
      for (int x = c_begin + lane; x < c_end; x += 32) cp_async4(smem_u32(tmp + x - c_begin), list.idx + list.at(x));
  }
  char* const qst = smem + kStageBytes;
  if (threadIdx.x == 0) {
    for (int x = 0; x < kQParts; ++x) mbar_init(&bars[kBarQLoad + x], 1);
    fence_barrier_init();
    for (int hd = 0, x = 0; hd < nh; hd += kQWarps, ++x) {
      const uint32_t bytes = (uint32_t)min(kQWarps, nh - hd) * kQPitch;
      mbar_arrive_expect_tx(&bars[kBarQLoad + x], bytes);
      bulk_load_g2s(smem_u32(qst + hd * kQPitch), reinterpret_cast<const char*>(qsrc) + hd * kQPitch, bytes, &bars[kBarQLoad + x]);
    }
  }
  if (threadIdx.x == 64) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars[kBarKvFull + s], kProducerWarps);
      mbar_init(&bars[kBarRows + s], 1);
      mbar_init(&bars[kBarKvEmpty + s], 1);
    }
    mbar_init(&bars[kBarSegFree], kProducerWarps);
    mbar_init(&bars[kBarSegFull], 1);
    mbar_init(&bars[kBarQReady], kQWarps);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars[kBarSFull + x], 1);
      mbar_init(&bars[kBarSFree + x], 2 * HB);      // the softmax warps that hold heads
      mbar_init(&bars[kBarAReady + x], 2 * HB);     // their references are known
      mbar_init(&bars[kBarPReady + x], 2 * HB + kFixWarps);   // their weights are written, O follows the references
      mbar_init(&bars[kBarPFree + x], 1);
    }
    mbar_init(&bars[kBarPvFinal], 1);
    mbar_init(&bars[kBarMmaFin], 1);
    mbar_init(&bars[kBarMmaFin2], 1);
    mbar_init(&bars[kBarNever], 1);         // nothing arrives: the stall test hook waits on it
    *abort_s = 0;
    for (int x = 0; x < 16; ++x) moved_s[x] = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_base_s, kTmemCols);
    tmem_relinquish();
  }
  if (warp == kProducerWarp && lane == 0) {
    prefetch_tmap(&tmap_lat);
    prefetch_tmap(&tmap_rope);
  }
  const int seq_len = p.seq_lens[b];
  const ShardSel sel = shard_sel(seq_len, seq_len - (p.Q - 1 - qi), r, p.n_splits, p.interleave);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_base_s;

  // ---- index resolution (warps 8-15): count per warp chunk, then ordered compaction ----
  int total = 0;
  int n_local = 0;                         // tiles
  auto count_tiles = [&]() { n_local = (total + kNt - 1) / kNt; };
  auto fail = [&](void) {
    give_up(p.status, abort_s);
  };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, wl));
  };

  // warps 0-7: warp 4 half + quad holds heads 16 quad + 8 half .. + 7 whole, a thread one of
  // them (row lane / 4 + 8 half of a 16-lane load), its reference (log2 units) and its share of
  // its sum; with 32 heads or fewer the warps of two quadrants hold none
  const int quad = warp & 3, half = warp >> 2;
  const int head = 16 * quad + 8 * half + (lane >> 2);
  const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
  float ref = -INFINITY, top = -INFINITY;   // reference of O; of the sums (the largest so far)
  float l_sum = 0.f, l_kept = 0.f;          // of the weights, and of the weights as they are stored
  // Roles follow in place, so that each warp runs through code that lies next to what it ran
  // before (the instruction cache is cold at every launch).
  if (warp >= kSoftWarps && warp < kFixWarp) {
    int row_r[8], cnt = 0;
    auto compact = [&](int* to, int at, int cap) {        // this round's rows from to[at] on; returns the next place
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const unsigned mask = __ballot_sync(0xffffffffu, row_r[k] >= 0);
        const int o = at + __popc(mask & lanemask_lt());
        if (row_r[k] >= 0 && o < cap) to[o] = row_r[k];
        at += __popc(mask);
      }
      return at;
    };
    if (staged) cp_wait_all();
#pragma unroll 1
    for (int j0 = c_begin; j0 < c_end; j0 += 256) {
      if (staged) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int j = j0 + 32 * k + lane;
          pos_r[k] = j < c_end ? tmp[j - c_begin] : -1;       // what this lane copied
        }
      } else if (!one_round) {
        load8(list, j0, c_end, lane, pos_r);
      }
      const int mine = resolve8<kInterleaved>(kp, pos_r, sel, bt_row, hg == 0, row_r);
      if (staged) cnt = compact(tmp, cnt, chunk); else cnt += __reduce_add_sync(0xffffffffu, mine);
    }
    if (lane == 0) wcount_s[warp - kSoftWarps] = cnt;
    named_barrier(4, 32 * kListWarps);
    int off = 0;
#pragma unroll
    for (int w = 0; w < kListWarps; ++w) {
      const int c = wcount_s[w];
      if (w < warp - kSoftWarps) off += c;
      total += c;
    }
    if (one_round) {
      if (c_begin < c_end) compact(list_s, off, kListCap);
    } else if (staged && total <= kListCap) {
      for (int o = lane; o < cnt; o += 32) list_s[off + o] = tmp[o];
    } else {
#pragma unroll 1
      for (int j0 = c_begin; j0 < c_end && off <= kListCap; j0 += 256) {
        int pos[8];
        load8(list, j0, c_end, lane, pos);
        resolve8<kInterleaved>(kp, pos, sel, bt_row, false, row_r);
        const int before = off;
        off = compact(list_s, off, kListCap);
        if (lane == 0 && before <= kListCap && off > kListCap) {   // (one round at most)
          seg_s[0] = j0;
          seg_s[1] = before;
        }
      }
    }
    // the last tile's missing rows: an index past the cache, which the gathers read as zeros
    if (warp == kSoftWarps)
      for (int o = total + lane; o < min((total + kNt - 1) / kNt * kNt, kListCap); o += 32) list_s[o] = kp.num_rows;
    // the gathers of the producer warps (async proxy) write over the staged list: every list warp's
    // accesses to it (generic proxy) come before them
    if (staged) fence_proxy_async_smem();
    named_barrier(4, 32 * kListWarps);
    if (lane == 0 && warp == kSoftWarps) wcount_s[kListWarps] = total;
    __syncwarp();
    asm volatile("bar.arrive %0, %1;" ::"r"(5), "r"(kThreads) : "memory");   // the other warps read `total`
    count_tiles();
    if (warp >= kProducerWarp && warp < kProducerWarp + kProducerWarps) {
      // =================== gathers ===================================================
      // Warp pw takes the tile's row groups pw, pw + 4, ... (4 rows each), five gather4 a group,
      // all from one lane: the lanes of a warp would issue theirs one after the other, each with
      // its operands moved to uniform registers first.  The warp waits for nothing but stages.
      const int pw = warp - kProducerWarp;
      constexpr int kGroupsOf = kNt / 4 / kProducerWarps;
      int seg = 0, n = 0;
      bool ok = true;
      for (; n < n_local && !*abort_s; ++n) {
        const int at = n % kStages;
        // stages 1 and 2 hold q until it is in TMEM; later tiles wait for P.V of the stage's last
        if (n > 0 && !(ok = n >= kStages ? wait_warp(&bars[kBarKvEmpty + at], ((n / kStages) - 1) & 1)
                                         : wait_warp(&bars[kBarQReady], 0)))
          break;
        const int first = kNt * n;
        if (first >= (seg + 1) * kListCap) {      // more valid entries than the list holds
          if (lane == 0) mbar_arrive(&bars[kBarSegFree]);
          if (!(ok = wait_warp(&bars[kBarSegFull], seg & 1))) break;
          ++seg;
        }
        const int* rows = list_s + (first - seg * kListCap) + 4 * pw;
        const uint32_t st = smem_u32(smem + at * kStageBytes);
        uint64_t* full = &bars[kBarKvFull + at];
        if (elect_one()) {
          mbar_arrive_expect_tx(full, kGroupsOf * 4 * kDQK);
  #pragma unroll
          for (int g = 0; g < kGroupsOf; ++g) {
            const int y = 4 * (pw + kProducerWarps * g);
            const int4 rr = *reinterpret_cast<const int4*>(rows + 4 * kProducerWarps * g);
  #pragma unroll
            for (int m = 0; m < 4; ++m)
              tma_gather4(st + m * kBlk + y * 128, &tmap_lat, 128 * m, rr.x, rr.y, rr.z, rr.w, full);
            tma_gather4(st + 4 * kBlk + y * 64, &tmap_rope, kDV, rr.x, rr.y, rr.z, rr.w, full);
          }
        }
        __syncwarp();
      }
      if (!ok) fail();
      // no gather of this CTA may still be landing in shared memory at exit
      for (int k = n > kStages ? n - kStages : 0; k < n; ++k)
        if (!__all_sync(0xffffffffu, wait_bar(&bars[kBarKvFull + k % kStages], (k / kStages) & 1, kDrainLimit, kLanded)))
          report_status(p.status, kStatusTimeout);
    } else if (warp == kRowWarp) {
      // =================== the rows' scales, and the rest of a long list ==============
      // Scales are single words anywhere in memory: those of the next two tiles are in flight
      // while two are published.  A segment of the list (64 tiles) begins with a
      // pair.
      constexpr int kAhead = 2, kPer = kNt / 32;
      static_assert(kListCap / kNt % kAhead == 0, "segments begin with a pair");
      float cur[kAhead][kPer], nxt[kAhead][kPer];
      int seg = 0, j = seg_s[0], ord = seg_s[1];   // the next segment's first round, entries before it
      bool ok = true;
      auto load4 = [&](int n0, float (&v)[kAhead][kPer]) {
  #pragma unroll
        for (int d = 0; d < kAhead; ++d) {
          const int* rows = list_s + kNt * (n0 + d) - seg * kListCap + lane;
  #pragma unroll
          for (int u = 0; u < kPer; ++u) {
            const int row = n0 + d < n_local ? rows[32 * u] : kp.num_rows;
            v[d][u] = row < kp.num_rows ? __ldg(kp.qp.scales + div_by(row, kp.gr_mul, kp.gr_shift)) : -1.f;
          }
        }
      };
      load4(0, cur);
  #pragma unroll 1
      for (int n0 = 0; n0 < n_local && ok && !*abort_s; n0 += kAhead) {
        const int first = kNt * (n0 + kAhead);
        const bool more = n0 + kAhead < n_local, turn = more && first >= (seg + 1) * kListCap;
        if (more && !turn) load4(n0 + kAhead, nxt);
  #pragma unroll
        for (int d = 0; d < kAhead; ++d) {
          const int n = n0 + d, at = n % kStages;
          if (n >= n_local || !ok) break;
          if (n >= kStages && !(ok = wait_warp(&bars[kBarKvEmpty + at], ((n / kStages) - 1) & 1))) break;
  #pragma unroll
          for (int u = 0; u < kPer; ++u) {
            // a row that does not exist (-1) has scale 0: weight 0.  One whose group was never
            // written (0) counts, with values of zero: its scale is the least one, and NaN stays
            const float c = cur[d][u] < 0.f ? 0.f : cur[d][u] < 0x1p-100f ? 0x1p-100f : cur[d][u];
            const int y = at * kNt + lane + 32 * u;
            float* rp = reinterpret_cast<float*>(rows_s) + 4 * (y >> 1) + (y & 1);
            rp[0] = c;
            rp[2] = __log2f(c);
            inv_s[y] = c > 0.f ? __frcp_rn(c) : 0.f;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kBarRows + at]);
        }
        if (turn && ok) {
          // once the producers have issued the segment's last tile, the next segment takes its
          // place (they only wait for tiles that are published by now)
          if (!(ok = wait_warp(&bars[kBarSegFree], seg & 1))) break;
          ++seg;
          const int base = seg * kListCap;
  #pragma unroll 1
          while (j < entries) {
            int pos[8], row[8], to = ord;
            load8(list, j, entries, lane, pos);
            resolve8<kInterleaved>(kp, pos, sel, bt_row, false, row);
  #pragma unroll
            for (int k = 0; k < 8; ++k) {
              const unsigned mask = __ballot_sync(0xffffffffu, row[k] >= 0);
              const int o = to + __popc(mask & lanemask_lt()) - base;
              if (row[k] >= 0 && o >= 0 && o < kListCap) list_s[o] = row[k];
              to += __popc(mask);
            }
            if (to > base + kListCap) break;       // the round goes on in the segment after
            ord = to;
            j += 256;
          }
          for (int o = total - base + lane; o < min(n_local * kNt - base, kListCap); o += 32) list_s[o] = kp.num_rows;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kBarSegFull]);
          load4(n0 + kAhead, nxt);
        }
  #pragma unroll
        for (int d = 0; d < kAhead; ++d)
  #pragma unroll
          for (int u = 0; u < kPer; ++u) cur[d][u] = nxt[d][u];
      }
      if (!ok) fail();
    } else if (warp == kQkWarp || warp == kPvWarp) {
      // =================== tcgen05 MMA issue: QK^T (warp 8) and P.V (warp 9) ========
      // (the whole warp walks the tiles and waits; one lane issues)
      if (n_local > 0) {
        bool ok = true;
        const uint32_t st0 = smem_u32(smem);
        if (warp == kQkWarp) {
          // test hook: a wait that cannot complete, so the wait limit runs out
          ok = !p.stall || wait_warp(&bars[kBarNever], 0);
          ok = ok && wait_warp(&bars[kBarQReady], 0);
          tc_fence_after();
          constexpr uint32_t id = idesc_e4m3(128, kNt, 0, 0);
          int s = 0;
          uint32_t full = 0;
          for (int n = 0; ok && n < n_local && !*abort_s; ++n) {
            const int sb = kSBufs == 2 ? n & 1 : 0;
            if (!(ok = wait_warp(&bars[kBarKvFull + s], full))) break;
            // the score buffer is free once the softmax has read the tile before from it
            if (n >= kSBufs && !(ok = wait_warp(&bars[kBarSFree + sb], (kSBufs == 2 ? (n >> 1) - 1 : n - 1) & 1))) break;
            tc_fence_after();
            const uint32_t st = st0 + s * kStageBytes;
            const uint32_t d = tmem + (sb ? kColS1 : kColS);
            if (elect_one()) {
              const uint32_t b0 = desc_lo(st, 16);
  #pragma unroll
              for (int k = 0; k < 16; ++k)
                mma8_ts<desc_hi(1024, kSwizzle128)>(d, tmem + kColQ + 8 * k, b0 + (((k >> 2) * kBlk + (k & 3) * 32) >> 4),
                                                    id, k > 0);
  #pragma unroll
              for (int k = 0; k < 2; ++k)
                mma8_ts<desc_hi(512, kSwizzle64)>(d, tmem + kColQ + 128 + 8 * k, b0 + ((4 * kBlk + k * 32) >> 4), id, 1);
              mma_commit(&bars[kBarSFull + sb]);
            }
            __syncwarp();
            if (++s == kStages) { s = 0; full ^= 1; }
          }
        } else {
          // A = E^T: columns 128m..128m+127 of 32 tile rows, MN-major (one SW128 atom wide);
          // B = P^T: NH heads x 32 rows, K-major.  The four blocks' accumulators alternate.
          int s = 0;
          for (int n = 0; ok && n < n_local && !*abort_s; ++n) {
            const int bb = n & 1;
            if (!(ok = wait_warp(&bars[kBarPReady + bb], (n >> 1) & 1))) break;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t a0 = desc_lo(st0 + s * kStageBytes, kBlk);
              const uint32_t b0 = desc_lo(st0 + kOffP + 2 * bb * kPBytes, 16);
  #pragma unroll
              for (int k = 0; k < kNt / 32; ++k)
  #pragma unroll
                for (int m = 0; m < 4; ++m) {
                  const uint32_t d = tmem + kColO + NH * m, a = a0 + ((m * kBlk + 4096 * k) >> 4), b = b0 + ((32 * k) >> 4);
                  const uint32_t id = idesc_e4m3_scaled(128, NH, 1, 0, k);
                  const uint32_t sf_e = tmem + kColSfE, sf_p = tmem + kColSfP + 4 * bb;
                  mma8_scaled_ss<desc_hi(1024, kSwizzle128), desc_hi(1024, kSwizzle128), true>(d, a, b, id, sf_e, sf_p,
                                                                                               k > 0 || n > 0);
                  mma8_scaled_ss<desc_hi(1024, kSwizzle128), desc_hi(1024, kSwizzle128), false>(
                      d, a, b + (kPBytes >> 4), id, sf_e, sf_p + 2, 1);
                }
              mma_commit(&bars[kBarKvEmpty + s]);
              mma_commit(&bars[kBarPFree + bb]);
              if (n == n_local - 1) mma_commit(&bars[kBarPvFinal]);
            }
            __syncwarp();
            if (++s == kStages) s = 0;
          }
        }
        if (!ok) fail();
        // every MMA this warp issued has completed before TMEM is released
        // (the same lane is elected every time: a commit covers its thread's MMAs)
        uint64_t* fin_bar = &bars[warp == kQkWarp ? kBarMmaFin : kBarMmaFin2];
        if (elect_one()) mma_commit(fin_bar);
        __syncwarp();
        if (!__all_sync(0xffffffffu, wait_bar(fin_bar, 0, kDrainLimit))) report_status(p.status, kStatusTimeout);
      }
    }
  } else {
    // ---- q as hi and lo e4m3 rows, a head a warp as it lands, in place in shared memory (stages
    // 1 and 2, which the gathers leave alone until q is ready); then to the TMEM lanes
#pragma unroll 1
    for (int hd = wq; hd < NH; hd += kQWarps) {
      if (hd < nh && !__all_sync(0xffffffffu, wait_bar(&bars[kBarQLoad + hd / kQWarps], 0, kDrainLimit)))
        report_status(p.status, kStatusTimeout);
      char* at = qst + hd * kQPitch;
      uint4 x[3];
#pragma unroll
      for (int k = 0; k < 3; ++k)
        x[k] = hd < nh && lane + 32 * k < 72 ? *reinterpret_cast<const uint4*>(at + 16 * (lane + 32 * k))
                                             : make_uint4(0, 0, 0, 0);
      uint32_t am2 = 0;                       // magnitudes of both halves
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        am2 = __vimax3_u16x2(am2, x[k].x & 0x7fff7fffu, x[k].y & 0x7fff7fffu);
        am2 = __vimax3_u16x2(am2, x[k].z & 0x7fff7fffu, x[k].w & 0x7fff7fffu);
      }
      const uint32_t am = __reduce_max_sync(0xffffffffu, max(am2 & 0xffffu, am2 >> 16));
      const bool bad = am >= 0x7f80u;       // an infinity or NaN: the head's result is NaN
      // 2^ke: the least power of two with amax / 2^ke <= 448
      int ke = (int)(am >> 7) - 135 + ((am & 0x7f) > 0x60 ? 1 : 0);
      ke = am < 0x80u || bad ? 0 : max(ke, -100);
      const float down = (p.scale < 0.f ? -1.f : 1.f) * __int_as_float((127 - ke) << 23);
      if (lane == 0)
        qc_s[hd] = bad ? __int_as_float(0x7fc00000)
                       : fmaxf(fabsf(p.scale) * kLog2e * __int_as_float((127 + ke) << 23), 1e-30f);
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // a scaled value has 8 bits below 2^9: f16 holds it (to 2^-24, below lo's 2^-13)
          const float a = __uint_as_float(w[i] << 16), c = __uint_as_float(w[i] & 0xffff0000u);
          const __half2 v = __floats2half2_rn(a * down, c * down);
          hi[i] = e4m3x2_h(v);
          lo[i] = e4m3x2_h(__hmul2(__hsub2(v, half2_of(hi[i])), __floats2half2_rn(16.f, 16.f)));
        }
        if (lane + 32 * k < 72) {
          char* to = at + 16 * q_word(hd, (lane + 32 * k) >> 1) + 8 * (lane & 1);
          *reinterpret_cast<uint2*>(to) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
          *reinterpret_cast<uint2*>(to + kDQK) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
        }
      }
    }
    named_barrier(1, 32 * kQWarps);
    const int quad = warp & 3;
    const int row = 16 * quad + (lane & 15);
    const char* mine = qst + row * kQPitch + (lane >= 16 ? kDQK : 0);
#pragma unroll 1
    for (int c = wq >> 2; c < 9 && quad < HB; c += kQWarps / 4) {     // 64 columns of q are 16 columns of TMEM
      uint32_t v[16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 x = *reinterpret_cast<const uint4*>(mine + 16 * q_word(row, 4 * c + k));
        v[4 * k] = x.x; v[4 * k + 1] = x.y; v[4 * k + 2] = x.z; v[4 * k + 3] = x.w;
      }
      tmem_st16(tmem + ((uint32_t)(quad * 32) << 16) + kColQ + 16 * c, v);
    }
    if (warp >= kFixWarp)                   // (warps 16-19 reach the lanes of all quadrants)
      tmem_st4(tmem + ((uint32_t)(quad * 32) << 16) + kColSfE, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
    tmem_st_wait();
    tc_fence_before();
    fence_proxy_async_smem();               // the gathers write these stages next
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[kBarQReady]);
    named_barrier(5, kThreads);
    total = wcount_s[kListWarps];
    count_tiles();
    if (warp < kSoftWarps) {
      // =================== softmax (warps 0-7) ======================================
      if (quad < HB) {
        float c_head = qc_s[head];
        const bool bad_q = c_head != c_head;
        if (bad_q) c_head = 1e-30f;
        const uint64_t c2 = pack2(c_head, c_head), sixteenth = pack2(0.0625f, 0.0625f);
        uint64_t l2 = 0, k2 = 0;                                // two running sums each
        // this head's row of P^T (K-major SW128) and this thread's bytes 16 k + 8 u + 2 (lane % 4)
        char* const p_row = smem + kOffP + head * 128 + 2 * (lane & 3);
        for (int i = 0; i < n_local; ++i) {
          const int bb = i & 1, sb = kSBufs == 2 ? bb : 0, st = i % kStages;
          if (*abort_s || !wait_warp(&bars[kBarSFull + sb], (kSBufs == 2 ? i >> 1 : i) & 1) ||
              !wait_warp(&bars[kBarRows + st], (i / kStages) & 1)) {
            fail();
            break;
          }
          tc_fence_after();
          // x = log2 of the weight: S = hi + lo / 16, then scale, head factor and log2 scale.
          // Pairs of rows 8 j + 2 (lane % 4), j < 12
          uint64_t x[kNt / 8];
          constexpr int kBatch = kNt / 32;                    // 16-row loads in flight at a time
          const uint32_t s_col = lane_base + (sb ? kColS1 : kColS);
          const float4* rs = rows_s + st * (kNt / 2) + (lane & 3);
          float mx[kNt / kWBlock] = {-INFINITY, -INFINITY, -INFINITY};   // of each 32 rows
  #pragma unroll
          for (int k3 = 0; k3 < kNt / 16; k3 += kBatch) {
            uint32_t vh[kBatch][8], vl[kBatch][8];
  #pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              tmem_ld_16x16(s_col + 16 * (k3 + k), vh[k]);
              tmem_ld_16x16(s_col + (16u << 16) + 16 * (k3 + k), vl[k]);
            }
            tmem_ld_wait();
            if (k3 + kBatch == kNt / 16) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars[kBarSFree + sb]);
            }
  #pragma unroll
            for (int k = 0; k < kBatch; ++k)
  #pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int j = 2 * (k3 + k) + u;
                const uint64_t hi = half ? pack2u(vh[k][4 * u + 2], vh[k][4 * u + 3]) : pack2u(vh[k][4 * u], vh[k][4 * u + 1]);
                const uint64_t lo = half ? pack2u(vl[k][4 * u + 2], vl[k][4 * u + 3]) : pack2u(vl[k][4 * u], vl[k][4 * u + 1]);
                const float4 cr = rs[4 * j];
                x[j] = fma2(fma2(lo, sixteenth, hi), mul2(pack2(cr.x, cr.y), c2), pack2(cr.z, cr.w));
                const float2 f = unpack2(x[j]);
                mx[j / 4] = fmaxf(mx[j / 4], fmaxf(f.x, f.y));
              }
          }
  #pragma unroll
          for (int o = 1; o < 4; o <<= 1)
  #pragma unroll
            for (int k = 0; k < kNt / kWBlock; ++k) mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], o));
          // P buffer bb, and its flags, factors and scales, are free once P.V of tile i-2 is done
          if (i >= 2 && !wait_warp(&bars[kBarPFree + bb], ((i >> 1) - 1) & 1)) {
            fail();
            break;
          }
          // A block's weights are stored under 2^e, its largest in (2^7, 2^8].  O's reference moves only
          // where a scale would be 2^kRise above it (and then those of the warp's heads that have risen)
          float e[kNt / kWBlock];
  #pragma unroll
          for (int k = 0; k < kNt / kWBlock; ++k) e[k] = ceilf(mx[k]) - kPeak;
          const float most = fmaxf(fmaxf(e[0], e[1]), e[2]);
          const bool moved = __any_sync(0xffffffffu, i > 0 && most > ref + kRise);
          const float ref_new = i == 0 || (moved && most > ref) ? most : ref;
          if (moved && (lane & 3) == 0) alpha_s[64 * bb + head] = ex2(ref - ref_new);
          ref = ref_new;
          uint32_t sf = 0;
  #pragma unroll
          for (int k = 0; k < kNt / kWBlock; ++k) {
            e[k] = fmaxf(e[k], ref - kFall);
            sf |= (uint32_t)((int)(e[k] - ref) + 127) << (8 * k);     // (a NaN, of a spoilt head, becomes 0)
          }
          if ((lane & 3) == 0) sf_s[64 * bb + head] = sf;
          if (lane == 0) moved_s[8 * bb + 2 * quad + half] = moved;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kBarAReady + bb]);
          // the sum's reference is the largest e so far
          const float top_new = fmaxf(top, most), fade = ex2(top - top_new);
          l2 = mul2(l2, pack2(fade, fade));
          k2 = mul2(k2, pack2(fade, fade));
          top = top_new;
          // P = 2^(x - e) as hi + lo / 16.  Into one sum goes p = P / scale; into another 16 times what the
          // rounding of a large weight added to its p (a small one may be off by more than itself, and
          // one of a small scale then by more than all others)
          const float2* iv = reinterpret_cast<const float2*>(inv_s + st * kNt) + (lane & 3);
          char* const row = p_row + 2 * bb * kPBytes;
  #pragma unroll
          for (int k = 0; k < kNt / kWBlock; ++k) {
            const uint64_t ne = pack2(-e[k], -e[k]);
            uint64_t sum = 0, more = 0;
  #pragma unroll
            for (int j = 4 * k; j < 4 * k + 4; ++j) {
              const float2 f = unpack2(add2(x[j], ne));
              const float p0 = ex2(f.x), p1 = ex2(f.y);
              const float2 inv = iv[4 * j];
              sum = fma2(pack2(p0, p1), pack2(inv.x, inv.y), sum);
              // 11 bits are enough under the 8 that hi and lo keep
              const __half2 w = __floats2half2_rn(p0, p1);
              const uint32_t hi = e4m3x2_h(w);
              const int at = (((j >> 1) ^ (head & 7)) << 4) + 8 * (j & 1);
              *reinterpret_cast<uint16_t*>(row + at) = (uint16_t)hi;
              const __half2 left = __hmul2(__hsub2(w, half2_of(hi)), __floats2half2_rn(16.f, 16.f));
              const uint32_t lo = e4m3x2_h(left);
              *reinterpret_cast<uint16_t*>(row + at + kPBytes) = (uint16_t)lo;
              const float2 d = __half22float2(__hmul2(__hsub2(half2_of(lo), left), __hge2(w, __floats2half2_rn(kFine, kFine))));
              more = fma2(pack2(d.x, d.y), pack2(inv.x, inv.y), more);
            }
            const float part = ex2(e[k] - top);
            l2 = fma2(sum, pack2(part, part), l2);
            k2 = fma2(more, pack2(part, part), k2);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kBarPReady + bb]);
        }
        const float2 f = unpack2(l2);
        l_sum = f.x + f.y;
        l_sum += __shfl_xor_sync(0xffffffffu, l_sum, 1);
        l_sum += __shfl_xor_sync(0xffffffffu, l_sum, 2);
        const float2 g = unpack2(k2);
        l_kept = g.x + g.y;
        l_kept += __shfl_xor_sync(0xffffffffu, l_kept, 1);
        l_kept += __shfl_xor_sync(0xffffffffu, l_kept, 2);
        l_kept = l_sum + l_kept * 0.0625f;
        if (bad_q && n_local > 0) l_sum = l_kept = __int_as_float(0x7fc00000);
      }
    } else if (warp >= kFixWarp) {
      // =================== O follows the references (warps 16-19) ====================
      // They put the scales of tile i's weights into TMEM while the softmax warps write the weights.
      // Where a head's reference moved with tile i, its column of O^T is scaled between P.V of
      // tiles i-1 and i.
      const uint32_t my_lanes = tmem + ((uint32_t)((warp - kFixWarp) * 32) << 16);
      for (int i = 0; i < n_local && !*abort_s; ++i) {
        const int bb = i & 1;
        if (!wait_warp(&bars[kBarAReady + bb], (i >> 1) & 1)) {
          fail();
          break;
        }
        {
          // the scales of the tile's weights; lo's are 2^-4 of hi's
          const volatile uint32_t* sp = sf_s + 64 * bb + lane;
          const uint32_t s0 = sp[0], s1 = NH == 64 ? sp[32] : s0;
          tmem_st4(my_lanes + kColSfP + 4 * bb, s0, s1, s0 - 0x040404u, s1 - 0x040404u);
        }
        uint64_t m8 = *reinterpret_cast<const volatile uint64_t*>(moved_s + 8 * bb);
        if (m8 != 0) {
          if (!wait_warp(&bars[kBarPFree + (bb ^ 1)], ((i - 1) >> 1) & 1)) {
            fail();
            break;
          }
          tc_fence_after();
  #pragma unroll 1
          while (m8 != 0) {
            const int oct = (__ffsll((long long)m8) - 1) >> 3;
            m8 &= m8 - 1;
            const float4 a = *reinterpret_cast<const float4*>(alpha_s + 64 * bb + 8 * oct);
            const float4 c = *reinterpret_cast<const float4*>(alpha_s + 64 * bb + 8 * oct + 4);
            const float al[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
            uint32_t o[32];
            const uint32_t at = my_lanes + kColO + 8 * oct;
  #pragma unroll
            for (int m = 0; m < 4; ++m) tmem_ld8(at + NH * m, o + 8 * m);
            tmem_ld_wait();
  #pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al[k & 7]);
  #pragma unroll
            for (int m = 0; m < 4; ++m) tmem_st8(at + NH * m, o + 8 * m);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kBarPReady + bb]);
      }
    }
  }

  // ---- merge of the cluster's partial results and the output ---------------------
  __syncwarp();
  if (warp < kSoftWarps) {
    if (n_local > 0 && !*abort_s && !wait_warp(&bars[kBarPvFinal], 0)) fail();
    if (quad < HB && (lane & 3) == 0) {
      ml_s[head] = make_float2(top, l_sum);
      below_s[head] = ref - top;
      kept_s[head] = l_kept;
      if (G == 1) scale_s[head] = l_kept != 0.f ? ex2(ref - top) / l_kept : 0.f;
    }
  }
  // (a CTA alone needs no cluster barrier, here and below)
  tc_fence_before();
  if (G > 1) cluster_sync(); else __syncthreads();   // every CTA's (m, l) is published and its stages are idle
  tc_fence_after();
  const bool good = !*abort_s, have_o = good && n_local > 0;
  const size_t lse_at = ((size_t)r * T + t) * p.h + h0, out_at = lse_at * kDV;   // nh rows of 512, one after the other
  const uint32_t my_lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  if (G == 1) {
    // O / l straight to global memory: every warp takes (column block, 16 heads) pieces of its
    // TMEM lanes, 32 columns of a head a store
    if (threadIdx.x < nh && good) {
      const float2 ml = ml_s[threadIdx.x];
      p.lse[lse_at + threadIdx.x] = ml.y != 0.f ? (ml.x + __log2f(ml.y)) * kLn2 : -INFINITY;
    }
#pragma unroll 1
    for (int c = warp >> 2; c < 4 * HB && good; c += kThreads / 128) {
      const int m = c / HB, hb = 16 * (c % HB);
      if (hb >= nh) continue;
      uint32_t o[16];
      if (have_o) tmem_ld16(my_lanes + kColO + 16 * c, o);
      float f[16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 sc = *reinterpret_cast<const float4*>(scale_s + hb + 4 * k);
        f[4 * k] = sc.x; f[4 * k + 1] = sc.y; f[4 * k + 2] = sc.z; f[4 * k + 3] = sc.w;
      }
      if (have_o) tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 16; ++k) f[k] = have_o ? __uint_as_float(o[k]) * f[k] : 0.f;
      // two columns of a head a store: even lanes take heads hb .. + 7, odd lanes the other 8
      const int odd = lane & 1, hd = hb + 8 * odd;
      const size_t at = out_at + (size_t)hd * kDV + 128 * m + 32 * (warp & 3) + (lane & 30);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? f[k] : f[k + 8], 1);
        const float2 v = odd ? make_float2(got, f[k + 8]) : make_float2(f[k], got);
        if (hd + k >= nh) continue;
        if (kp.qp.out_bf16)
          *reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<__nv_bfloat16*>(p.out) + at + k * kDV) =
              __floats2bfloat162_rn(v.x, v.y);
        else
          *reinterpret_cast<float2*>(p.out + at + k * kDV) = v;
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
    return;
  }
  // Every thread of every CTA of the cluster reaches both cluster barriers.
  if (threadIdx.x < NH) {
    // this head's largest reference M, sum L and the weight of this CTA's O
    const int hd = threadIdx.x;
    float M = -INFINITY, L = 0.f, K = 0.f;
    for (uint32_t c = 0; c < G; ++c) M = fmaxf(M, ld_cluster_f32(mapa(&ml_s[hd], c)));
    for (uint32_t c = 0; c < G; ++c) {
      const uint32_t a = mapa(&ml_s[hd], c);
      const float lc = ld_cluster_f32(a + 4u);
      if (lc == 0.f) continue;
      const float f = ex2(ld_cluster_f32(a) - M);
      L += f * lc;
      K += f * ld_cluster_f32(mapa(&kept_s[hd], c));
    }
    const float2 mine = ml_s[hd];
    scale_s[hd] = mine.y != 0.f ? ex2(mine.x - M + below_s[hd]) / K : 0.f;
    if (crank == 0 && hd < nh && good) p.lse[lse_at + hd] = L != 0.f ? (M + __log2f(L)) * kLn2 : -INFINITY;
  }
  __syncthreads();
  // 32-column segment 4m + quad of O goes to CTA (4m + quad) / segs, into its idle stages, slot
  // of this CTA: [head][32 columns], so that a store is 128 bytes in one place (as 16 bytes a lane,
  // in 32 places, the exchange of 64 heads took several us)
  const int segs = 16 >> g_shift;
  float* recv = reinterpret_cast<float*>(smem);
#pragma unroll 1
  for (int c = warp >> 2; c < 4 * HB; c += kThreads / 128) {
    const int m = c / HB, hb = 16 * (c % HB), sg = 4 * m + (warp & 3);
    if (hb >= nh) continue;
    uint32_t o[16];
    if (have_o) {
      tmem_ld16(my_lanes + kColO + 16 * c, o);
      tmem_ld_wait();
    }
    const uint32_t dst = mapa(recv + ((size_t)(crank * segs + (sg & (segs - 1))) * NH + hb) * 32 + lane, sg / segs);
#pragma unroll
    for (int k = 0; k < 16; ++k)
      st_cluster_f32(dst + 128u * k, have_o ? __uint_as_float(o[k]) * scale_s[hb + k] : 0.f);
  }
  tc_fence_before();
  cluster_sync();   // every CTA's scaled partial O has landed with its owner
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
  if (!good) return;
  // this CTA's segments: the sum of the G scaled partials, in the order of the CTAs
  for (int x = warp; x < segs * (NH / 4); x += kThreads / 32) {
    const int sg = x & (segs - 1), k4 = x / segs;
    if (4 * k4 >= nh) break;
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    const float* src = recv + ((size_t)sg * NH + 4 * k4) * 32 + lane;
    for (uint32_t c = 0; c < G; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] += src[(size_t)c * segs * NH * 32 + 32 * k];
    const size_t at = out_at + 32 * ((int)crank * segs + sg) + lane;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (4 * k4 + k >= nh) break;
      if (kp.qp.out_bf16)
        reinterpret_cast<__nv_bfloat16*>(p.out)[at + (size_t)(4 * k4 + k) * kDV] = __float2bfloat16_rn(f[k]);
      else
        p.out[at + (size_t)(4 * k4 + k) * kDV] = f[k];
    }
  }
}

template <int NH, bool kIL>
constexpr auto q8_kernel() {
  return decode_q8_kernel<NH, kIL>;
}

// the cache as [num_rows, 576] bytes; one box = `cols` columns of one row (gathered four at a time)
bool make_rows_map(CUtensorMap* m, const void* kv8, int num_rows, int cols, CUtensorMapSwizzle swizzle) {
  typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::once_flag once;
  static EncodeFn fn = nullptr;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(ptr);
  });
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)kDQK, (cuuint64_t)num_rows};
  const cuuint64_t strides[1] = {(cuuint64_t)kDQK};
  const cuuint32_t box[2] = {(cuuint32_t)cols, 1}, es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(kv8), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

void launch_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, long long units, int G, cudaStream_t stream) {
  memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3((unsigned)(units * G), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = (unsigned)G;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
}

// once a device: the kernels' shared memory, and how many clusters of 2, 4 and 8 CTAs run at once
// (fewer than the SMs would hold: a cluster stays within one group of SMs)
cudaError_t prepare_decode_q8(int (&fit)[3]) {
  static std::atomic<bool> ready[64];
  static int fits[64][3];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    static std::mutex once;
    const std::lock_guard<std::mutex> hold(once);
    for (auto kernel : {q8_kernel<32, false>(), q8_kernel<32, true>(), q8_kernel<64, false>(), q8_kernel<64, true>()}) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
      if (e != cudaSuccess) return e;
    }
    for (int k = 0; k < 3 && !ready[dev].load(std::memory_order_relaxed); ++k) {
      cudaLaunchConfig_t cfg;
      cudaLaunchAttribute attr[1];
      launch_config(cfg, attr, 1, 2 << k, 0);
      e = cudaOccupancyMaxActiveClusters(&fits[dev][k], q8_kernel<64, false>(), &cfg);
      if (e != cudaSuccess) return e;
    }
    ready[dev].store(true, std::memory_order_release);
  }
  for (int k = 0; k < 3; ++k) fit[k] = fits[dev][k];
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_decode_q8(const DecodeQ8Params& qp, cudaStream_t stream) {
  const DecodeParams& p = qp.p;
  const long long T = (long long)p.B * p.Q;
  if (T == 0) return cudaSuccess;
  int fit[3];
  cudaError_t e = prepare_decode_q8(fit);
  if (e != cudaSuccess) return e;
  Q8Params kp;
  kp.qp = qp;
  kp.groups = (p.h + kGroupHeads - 1) / kGroupHeads;
  kp.group_heads = (p.h + kp.groups - 1) / kp.groups;
  const long long units = T * p.n_splits * kp.groups;
  // A unit is shared by up to 8 CTAs while all clusters run at once and there is more than a tile of
  // the list for each of half as many (three tiles for the first split).  9 tokens x 16 heads x 2048
  // rows, by 1, 2, 4, 8 CTAs: 33, 22, 16, 13 us; 64 heads 41, 29, 22, 19; 300 rows 12, 11, 10, 11 and
  // 15, 16, 15, 16; 180 rows 9.4, 10.1, 9.7, 10.2.  (38 units by 4 CTAs, which do not run at once: 32 us,
  // by 2: 23.)
  int G = 1;
  for (int k = 0; k < 3 && units <= fit[k] && p.top_k > (G > 2 ? G : 3) * kNt; ++k) G *= 2;
  if (units * G > 0x7fffffffLL) return cudaErrorInvalidValue;
  const bool il = p.interleave > 0 && p.n_splits > 1;
  // 32 padded heads or 64: 100 tokens x 32 heads x 2048 rows 39.8 us, as 64 heads 41.8; 4 tokens 15.7, 22.2
  auto kernel = kp.group_heads <= 32 ? (il ? q8_kernel<32, true>() : q8_kernel<32, false>())
                                     : (il ? q8_kernel<64, true>() : q8_kernel<64, false>());
  CUtensorMap lat, rope;
  kp.num_rows = p.num_blocks * p.block_size;
  divisor(p.block_size, kp.bs_mul, kp.bs_shift);
  divisor(qp.group, kp.gr_mul, kp.gr_shift);
  divisor((int)T, kp.T_mul, kp.T_shift);
  divisor(p.Q, kp.Q_mul, kp.Q_shift);
  if (!make_rows_map(&lat, p.kv, kp.num_rows, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_rows_map(&rope, p.kv, kp.num_rows, 64, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  launch_config(cfg, attr, units, G, stream);
  e = cudaLaunchKernelEx(&cfg, kernel, lat, rope, kp);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sfa
