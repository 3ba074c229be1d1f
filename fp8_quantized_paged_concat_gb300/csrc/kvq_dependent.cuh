// kvq_dependent.cuh -- dependent launches: a kernel that is set up while the
// one before it in the stream still runs.
//
// Every thread of such a kernel calls wait_for_previous() before its first
// access to memory (tensor memory among it, which a CTA before it may still
// have to take), on every path: so a kernel ends after the one before it, and
// what a stream orders stays ordered along a chain of them.  Measured, the
// same call queued from Python over and over: a single-token attention 8.2 ->
// 7.0 us, a compaction of one layer 6.2 -> 3.4, of 32 layers 15.1 -> 13.1, a
// tree of one user 20.5 -> 16.3; in a graph 0 to 0.4 us less.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace kvq {
namespace {

// The next kernel of the stream may be set up once every CTA has said so or left.
__device__ __forceinline__ void allow_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Returns when the kernels before are complete and their writes visible.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A load of what a kernel before may have written.  A plain one: the compiler
// may move a load through the read-only path (__ldg) up past the wait, and
// that path promises nothing for data written while the kernel is resident.
template <class T>
__device__ __forceinline__ T load_global(const T* p) {
  return *p;
}
// The same, opaque, where registers are short: plain loads of an unrolled loop
// are merged and held (mask words in the few-row attention's blocks of 16
// rows at head size 128: 80 bytes of spill loads a thread, 28 with opaque ones;
// 128 requests x 2048 keys 99.7 against 96.1 us, as trees 103 against 96; its
// blocks of 8 take the same time either way).
__device__ __forceinline__ uint64_t load_global64(const uint64_t* p) {
  uint64_t v;
  asm volatile("ld.global.b64 %0, [%1];" : "=l"(v) : "l"(p));
  return v;
}

// Launches kernel(args...) as a dependent one; cluster > 1: in clusters of that many CTAs (along x).
template <class... Params, class... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, int smem, int cluster,
                             cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t config = {};
  config.gridDim = grid;
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  config.attrs = at;
  config.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&config, kernel, static_cast<Params>(args)...);
}

}  // namespace
}  // namespace kvq
