// ptx_more.cuh -- further wrappers of PTX instructions and launches, for the kernels
// of the layer of experts and the prompt attention.  ptx.cuh holds those that the
// projections' kernels use: bench.py knows their measured traffic by a hash of their
// sources, that header among them.
#pragma once

#include "ptx.cuh"

namespace rnl {

// True on one lane of a converged warp.  What the branch behind it uses can stay in
// the warp's uniform registers, which the tensor-core instructions take their
// operands from; behind a test of the lane number each operand is moved there
// first, about 60 cycles an instruction.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// mbar_arrive_cluster for a hand-over that orders shared memory only (after a proxy
// fence): a release at cluster scope also waits for the CTA's traffic to global memory,
// about 1 us, which a hand-over per k-block cannot afford.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Launches a kernel that begins with grid_dependency_wait as a programmatic dependent
// of the one before it in the stream.  What the kernel before may have written
// is read by plain loads (or ld.cg) behind that wait: the read-only path (__ldg,
// ld.global.nc) is for data that nobody writes while the kernel is there, which a
// dependent is before its predecessor has ended, and such a load need not stay
// behind the wait.  Small kernels let the next one start behind
// their own wait: with the trigger in front of it, kernels pile up behind a long
// one and hold its SMs' places (16 tokens through a layer of experts in MXFP8: 147
// against 140 us, 141 without a trigger).
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t s,
                                    A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

// 16 bytes from global to shared memory without a register between; bytes 0
// reads nothing and writes zeros.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Arrives once on a barrier of this CTA when the copies that this thread has
// issued so far have landed (the barrier's count includes the arrival).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// 5-D tiled load with the completion in the pair's even CTA.
__device__ __forceinline__ void tma_load_5d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster,
                                                 int32_t c0, int32_t c1, int32_t c2, int32_t c3, int32_t c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// As tmem_st_4cols, 16 columns.
__device__ __forceinline__ void tmem_st_16cols(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

}  // namespace rnl
