// sfa_tree_simt.cu -- the attention of a tree of drafted tokens on CUDA cores, every shape: one CTA
// per (token, group of 8 heads).  The plain form of the definition, to cross-check the tensor cores'
// kernel.  Bound: fp32 arithmetic and shared-memory reads of q, and for few tokens the chain of four warps
// that take a position after the other: 6 nodes x 4 heads x 200 positions 74 us (tensor cores: 27; it is
// ahead at one position, 9 us).
#include <atomic>

#include "sfa_tree.cuh"

namespace sfa {
namespace {

constexpr int kHeads = 8;   // of a CTA

__global__ void __launch_bounds__(kTreeSimtWarps * 32) decode_tree_simt_kernel(const TreeParams p) {
  extern __shared__ float smem[];
  tree_simt<kHeads>(p, blockIdx.x, blockIdx.y * kHeads, smem);
}

}  // namespace

cudaError_t launch_decode_tree_simt(const TreeParams& p, cudaStream_t stream) {
  if (p.T == 0 || p.B == 0) return cudaSuccess;
  static std::atomic<bool> attr_set[64];   // per device: set once (a repeat is harmless)
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(decode_tree_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, tree_simt_smem(kHeads));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true, std::memory_order_release);
  }
  const dim3 grid(p.T, (p.h + kHeads - 1) / kHeads);
  decode_tree_simt_kernel<<<grid, kTreeSimtWarps * 32, tree_simt_smem(kHeads), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace sfa
