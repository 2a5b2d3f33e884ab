// Shared pieces of the operators around the layer (block norms, balance loss, optimiser):
// launches, asynchronous copies, arithmetic on pairs, sums over a block.
#pragma once

#include <atomic>

#include "common.cuh"

namespace moe {

void count_launch();
int num_sms();

// Allows kernel KERN `bytes` of dynamic shared memory, once a device (at every call it would
// cost a launch 0.5 us; after a cudaDeviceReset the launch fails, and the call says so).
template <auto KERN>
static cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  err = cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
  return err;
}

inline bool ptr_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline moe_status status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// Every kernel here is launched early: its blocks come up as the last ones of the kernel
// before it on the stream (of any origin) leave the SMs, and wait there for that kernel's end
// and its writes.  It saves a call 2 us (balance of 16384 x 256: 17.1 to 14.8 us, norm of
// 8121 x 2048: 20.7 to 18.6 us, calls one after another).  A kernel waits before it touches
// memory and only then lets the next one come up, so that a kernel that has begun knows that
// everything before its predecessor is done.  (The step of fp32 moments lets nothing come up.)
// The exception is the balance loss's join: it reads the sequence offsets, which its
// predecessor, the loss's own first kernel, only reads too, and may set the status before it
// waits.  What a predecessor writes must not be reached through __restrict__ pointers or
// read-only loads: both say that memory does not change while a kernel is resident.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... Params, typename... Args>
static cudaError_t launch_early_clusters(void (*kern)(Params...), dim3 grid, dim3 block, int smem, cudaStream_t s, int cluster, const Args&... args) {
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;    // of blocks along x, where it is not 0
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
  if (err == cudaSuccess) count_launch();
  return err;
}
template <typename... Params, typename... Args>
static cudaError_t launch_early(void (*kern)(Params...), dim3 grid, dim3 block, int smem, cudaStream_t s, const Args&... args) {
  return launch_early_clusters(kern, grid, block, smem, s, 0, args...);
}

// Asynchronous copies of 16, 8 or 4 bytes from global to shared memory, in groups.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most N of this thread's groups are under way.
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Two fp32 values in a register pair, and arithmetic on both in one instruction (rounded
// as two scalar ones, except that a mul2 whose only use is an add2 may become one fma2).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float x, float y) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpair(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Rounded down.
__device__ __forceinline__ f32x2 fma2_down(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ float sum_pair(f32x2 v) {
  const float2 f = unpair(v);
  return f.x + f.y;
}
// 1 / x within a unit; 0 where that is below fp32's normal numbers, infinite where x is.
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Eight consecutive elements, rounded once from fp32.
__device__ __forceinline__ void store8(moe_bf16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Sums of N values over a warp (WARP) or over the block, in a fixed order; every thread
// gets them.  `buf`: 32 * N floats of shared memory that the previous sum did not use (two
// buffers taken in turn need one barrier a sum).
template <bool WARP, int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float* buf) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], off);
  }
  if (WARP) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[warp * N + i] = s[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = lane < warps ? buf[lane * N + i] : 0.0f;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], off);
  }
}

}  // namespace moe
