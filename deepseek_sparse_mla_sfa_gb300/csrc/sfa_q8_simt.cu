// sfa_q8_simt.cu -- CUDA-core path of sparse MLA decode over the 8-bit latent cache: the
// plain definition, any shape, used to cross-check the tensor-core kernel
// (sfa_set_kernel_path(1)).
//
// One CTA per (query token, shard, group of 8 heads); its 4 warps take the selected
// entries round-robin with an online softmax each (running max m, sum l, output o, all
// fp32) and their states are joined at the end.  A row is dequantised to fp32 in registers
// (e4m3 * scale of its group is exact there for power-of-two scales).  Bound by the
// arithmetic: rows are read again for every 8 heads (64 tokens x 128 heads x 2048 rows: 4957 us,
// the tensor-core kernel 45).
#include <cuda_fp8.h>

#include "sfa_internal.h"

namespace sfa {
namespace {

constexpr int kHG = 8, kWarps = 4;
constexpr int kPairs = kDQK / 64;    // 9 pairs of columns a lane
constexpr int kVPairs = kDV / 64;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// the largest of the warps' maxima; NaN, which fmaxf passes over, where one of them is NaN
__device__ __forceinline__ float join_max(const float (&m)[kWarps][kHG], int hh) {
  float M = m[0][hh];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) M = m[w][hh] != m[w][hh] ? m[w][hh] : M != M ? M : fmaxf(M, m[w][hh]);
  return M;
}

__global__ void __launch_bounds__(kWarps * 32) decode_q8_simt_kernel(const DecodeQ8Params qp) {
  const DecodeParams& p = qp.p;
  __shared__ float q_s[kHG * kDQK];
  __shared__ float o_s[kHG * kDV];
  __shared__ float m_s[kWarps][kHG], l_s[kWarps][kHG];
  const int t = blockIdx.x, r = blockIdx.y, h0 = blockIdx.z * kHG;
  const int T = p.B * p.Q, nh = min(kHG, p.h - h0), b = t / p.Q;
  const int seq_len = p.seq_lens[b];
  const ShardSel sel = shard_sel(seq_len, seq_len - (p.Q - 1 - t % p.Q), r, p.n_splits, p.interleave);
  const int bt_row = p.bt_per_token ? t : b;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int x = threadIdx.x; x < kHG * kDQK; x += blockDim.x)
    q_s[x] = x / kDQK < nh ? __bfloat162float(p.q[((size_t)t * p.h + h0) * kDQK + x]) : 0.f;
  for (int x = threadIdx.x; x < kHG * kDV; x += blockDim.x) o_s[x] = 0.f;
  __syncthreads();

  float m[kHG], l[kHG], o[kHG][2 * kVPairs];
#pragma unroll
  for (int hh = 0; hh < kHG; ++hh) {
    m[hh] = -INFINITY;
    l[hh] = 0.f;
#pragma unroll
    for (int c = 0; c < 2 * kVPairs; ++c) o[hh][c] = 0.f;
  }
  const uint8_t* kv = reinterpret_cast<const uint8_t*>(p.kv);
  for (int j = warp; j < p.top_k; j += kWarps) {
    const int pos = p.topk_idx[(size_t)t * p.top_k + j];
    if (!sel.has(pos)) continue;
    const int blk = pos / p.block_size;
    const int phys = blk < p.max_blocks ? p.block_table[(size_t)bt_row * p.max_blocks + blk] : -1;
    if (phys < 0 || phys >= p.num_blocks) {
      if (lane == 0) report_status(p.status, kStatusBadBlock);
      continue;
    }
    const size_t row = (size_t)phys * p.block_size + pos % p.block_size;
    const float sc = qp.scales[row / qp.group];
    const uint16_t* src = reinterpret_cast<const uint16_t*>(kv + row * kDQK);
    float kx[2 * kPairs];
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(src[lane + 32 * k], __NV_E4M3);
      const float2 f = __half22float2(__half2(hr));
      kx[2 * k] = f.x * sc;
      kx[2 * k + 1] = f.y * sc;
    }
#pragma unroll
    for (int hh = 0; hh < kHG; ++hh) {
      if (hh >= nh) break;
      const float* qh = q_s + hh * kDQK;
      float part = 0.f;
#pragma unroll
      for (int k = 0; k < kPairs; ++k)
        part += qh[2 * lane + 64 * k] * kx[2 * k] + qh[2 * lane + 1 + 64 * k] * kx[2 * k + 1];
      const float s = warp_sum(part) * p.scale;
      const float m_new = s != s ? s : fmaxf(m[hh], s);   // a NaN score makes its head NaN
      const float alpha = expf(m[hh] - m_new), e = expf(s - m_new);
      l[hh] = l[hh] * alpha + e;
#pragma unroll
      for (int c = 0; c < 2 * kVPairs; ++c) o[hh][c] = o[hh][c] * alpha + e * kx[c];
      m[hh] = m_new;
    }
  }
#pragma unroll
  for (int hh = 0; hh < kHG; ++hh)
    if (lane == 0) {
      m_s[warp][hh] = m[hh];
      l_s[warp][hh] = l[hh];
    }
  __syncthreads();
  // the warps add their outputs, weighted to the common maximum, one after the other (a
  // fixed order: the same inputs give the same sums)
  for (int w = 0; w < kWarps; ++w) {
    if (warp == w) {
#pragma unroll
      for (int hh = 0; hh < kHG; ++hh) {
        const float M = join_max(m_s, hh);
        const float f = m[hh] == -INFINITY ? 0.f : expf(m[hh] - M);
#pragma unroll
        for (int c = 0; c < 2 * kVPairs; ++c) o_s[hh * kDV + 2 * lane + 64 * (c >> 1) + (c & 1)] += o[hh][c] * f;
      }
    }
    __syncthreads();
  }
  const size_t at = ((size_t)r * T + t) * p.h + h0;
  for (int x = threadIdx.x; x < nh * kDV; x += blockDim.x) {
    const int hh = x / kDV;
    const float M = join_max(m_s, hh);
    float lsum = 0.f;
    if (M != -INFINITY)
      for (int w = 0; w < kWarps; ++w) lsum += l_s[w][hh] * expf(m_s[w][hh] - M);
    const float val = M == -INFINITY ? 0.f : o_s[x] / lsum;
    if (qp.out_bf16)
      reinterpret_cast<__nv_bfloat16*>(p.out)[at * kDV + x] = __float2bfloat16_rn(val);
    else
      p.out[at * kDV + x] = val;
    if (x % kDV == 0) p.lse[at + hh] = M == -INFINITY ? -INFINITY : M + logf(lsum);
  }
}

}  // namespace

cudaError_t launch_decode_q8_simt(const DecodeQ8Params& qp, cudaStream_t stream) {
  const DecodeParams& p = qp.p;
  const int T = p.B * p.Q;
  if (T == 0) return cudaSuccess;
  decode_q8_simt_kernel<<<dim3(T, p.n_splits, (p.h + kHG - 1) / kHG), kWarps * 32, 0, stream>>>(qp);
  return cudaGetLastError();
}

}  // namespace sfa
