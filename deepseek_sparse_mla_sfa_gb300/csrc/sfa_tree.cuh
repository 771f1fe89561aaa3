// sfa_tree.cuh -- the attention of a tree of drafted tokens: its problem as the kernels see it, and
// one (token, group of heads) of it on CUDA cores.
#pragma once

#include "sfa_internal.h"

namespace sfa {

// the request of token t: the last b with token_start[b] <= t, -1 for a token of none (token_start
// ascends; an equal pair is a request without nodes)
__device__ __forceinline__ int tree_request(const int32_t* token_start, int B, int t) {
  if (B < 1 || t < token_start[0] || t >= token_start[B]) return -1;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (token_start[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// positions that a row of the block table reaches
__device__ __forceinline__ long long tree_reach(const TreeParams& p) { return (long long)p.max_blocks * p.block_size; }

constexpr int kTreeSimtWarps = 4;
constexpr int tree_simt_smem(int heads) {
  return 4 * (heads * kDQK + kTreeSimtWarps * heads * kDV + 2 * kTreeSimtWarps * heads);
}

__device__ __forceinline__ void tree_store(const TreeParams& p, size_t at, float v) {
  if (p.out_bf16)
    static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(v);
  else
    static_cast<float*>(p.out)[at] = v;
}

// Heads [h0, h0 + kHG) of token t, the first 128 threads of the CTA: its warps take the positions by
// turns, each with an online softmax (maximum, sum, output) a head, and join at the end.  A position
// that the token does not attend to is never read.
template <int kHG>
__device__ __forceinline__ void tree_simt(const TreeParams& p, int t, int h0, float* smem) {
  constexpr int kWarps = kTreeSimtWarps, kQK = kDQK / 64, kV = kDV / 64;
  float* q_s = smem;                                  // [kHG][576]
  float* o_s = q_s + kHG * kDQK;                      // [kWarps][kHG][512]
  float* m_s = o_s + kWarps * kHG * kDV;              // [kWarps][kHG]
  float* l_s = m_s + kWarps * kHG;                    // [kWarps][kHG]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = tree_request(p.token_start, p.B, t);
  if (b < 0) return;
  const int first = max(p.token_start[b], 0);
  const int n = min(min(p.token_start[b + 1], p.T) - first, p.max_nodes);
  if (t - first >= n) {
    if (threadIdx.x == 0) report_status(p.status, kStatusBadTree);
    return;
  }
  const int cached = max(p.cached[b], 0);
  const int nh = min(kHG, p.h - h0);
  const long long* mask = p.mask + (size_t)t * p.words;
  const int32_t* table = p.block_table + (size_t)b * p.max_blocks;
  for (int x = threadIdx.x; x < kHG * kDQK; x += kWarps * 32) {
    const int hh = x / kDQK, d = x % kDQK;
    q_s[x] = hh < nh ? __bfloat162float(p.q[((size_t)t * p.h + h0 + hh) * kDQK + d]) : 0.f;
  }
  __syncthreads();

  float m[kHG], l[kHG], o[kHG][2 * kV];
#pragma unroll
  for (int hh = 0; hh < kHG; ++hh) {
    m[hh] = -INFINITY;
    l[hh] = 0.f;
#pragma unroll
    for (int c = 0; c < 2 * kV; ++c) o[hh][c] = 0.f;
  }
  for (long long pos = warp; pos < (long long)cached + n; pos += kWarps) {
    if (pos >= tree_reach(p) && pos + kWarps < cached) pos += (cached - 1 - pos) / kWarps * kWarps;   // no blocks there
    if (pos >= cached) {
      const int j = (int)(pos - cached);
      if (!(mask[j / 64] >> (j % 64) & 1)) continue;
    }
    const long long blk = pos / p.block_size;
    const int phys = blk < p.max_blocks ? table[blk] : -1;
    if (phys < 0 || phys >= p.num_blocks) {
      if (lane == 0) report_status(p.status, kStatusBadBlock);
      continue;
    }
    const __nv_bfloat162* row =
        reinterpret_cast<const __nv_bfloat162*>(p.kv + ((size_t)phys * p.block_size + pos % p.block_size) * kDQK);
    float kx[2 * kQK];
#pragma unroll
    for (int k = 0; k < kQK; ++k) {
      const float2 f = __bfloat1622float2(row[lane + 32 * k]);
      kx[2 * k] = f.x;
      kx[2 * k + 1] = f.y;
    }
#pragma unroll
    for (int hh = 0; hh < kHG; ++hh) {
      if (hh >= nh) break;
      const float* qh = q_s + hh * kDQK;
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kQK; ++k) s += qh[2 * lane + 64 * k] * kx[2 * k] + qh[2 * lane + 1 + 64 * k] * kx[2 * k + 1];
#pragma unroll
      for (int u = 16; u > 0; u >>= 1) s += __shfl_xor_sync(0xffffffffu, s, u);
      s *= p.scale;
      const float m_new = fmaxf(m[hh], s);
      const float alpha = m[hh] == m_new ? 1.f : __expf(m[hh] - m_new);
      // a score of -inf has no weight; one that is NaN or +inf makes the sums NaN
      const float e = m_new == -INFINITY && s == s ? 0.f : __expf(s - m_new);
      l[hh] = l[hh] * alpha + e;
#pragma unroll
      for (int c = 0; c < 2 * kV; ++c) o[hh][c] = o[hh][c] * alpha + e * kx[c];
      m[hh] = m_new;
    }
  }
#pragma unroll
  for (int hh = 0; hh < kHG; ++hh) {
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      o_s[(warp * kHG + hh) * kDV + 2 * lane + 64 * k] = o[hh][2 * k];
      o_s[(warp * kHG + hh) * kDV + 2 * lane + 1 + 64 * k] = o[hh][2 * k + 1];
    }
    if (lane == 0) {
      m_s[warp * kHG + hh] = m[hh];
      l_s[warp * kHG + hh] = l[hh];
    }
  }
  __syncthreads();
  const size_t row0 = (size_t)t * p.h + h0;
  for (int x = threadIdx.x; x < nh * kDV; x += kWarps * 32) {
    const int hh = x / kDV, c = x % kDV;
    float M = -INFINITY, val = 0.f, lsum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, m_s[w * kHG + hh]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float lw = l_s[w * kHG + hh];
      if (lw == 0.f) continue;                 // (a warp without a position)
      const float sc = m_s[w * kHG + hh] == M ? 1.f : __expf(m_s[w * kHG + hh] - M);
      lsum += lw * sc;
      val += o_s[(w * kHG + hh) * kDV + c] * sc;
    }
    const bool none = lsum == 0.f;
    tree_store(p, (row0 + hh) * kDV + c, none ? 0.f : val / lsum);
    if (c == 0) p.lse[row0 + hh] = none ? -INFINITY : M + logf(lsum);
  }
  __syncthreads();
}

}  // namespace sfa
