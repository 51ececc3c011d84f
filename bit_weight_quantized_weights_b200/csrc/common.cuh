// Shared device helpers for the wq kernels (sm_100a only).
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <atomic>

#include "../../include/wq.h"

#if defined(__CUDA_ARCH__) && (__CUDA_ARCH__ < 1000)
#error "wq kernels are written for sm_100a only"
#endif

namespace wq {

// The 16 NF4 code values, passed to kernels by value (64 bytes of parameter
// space), so no device-global table has to be initialised.
struct Nf4Table {
  float v[16];
};

// Host: the table computed once per process from the QLoRA construction.
const Nf4Table& nf4_table();

// Wait control of the kernels with bounded mbarrier waits, passed by value.
//   limit_ns  how long any one wait may last before the kernel gives up
//   stall     test hook: when 1, the TMA producer withholds the loads of the
//             first k-tile, so the first waits on them expire (exercises the
//             timeout, abort and drain path without a device fault)
struct WaitCtl {
  uint64_t limit_ns;
  int32_t stall;
};

// Host: the process-wide setting (set by wq_test_set_wait; 2 s, no stall by
// default).
WaitCtl wait_ctl();
constexpr uint64_t sm100_default_wait_ns() { return 2000000000ull; }

// Host-side helpers shared by the launch wrappers.
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline wq_status launch_status() {
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}

// Programmatic dependent launch: the kernel may be set up while the one before it
// in the stream still runs, and begins with follow_previous() (or a wait of its own).
// A kernel of a few microseconds saves about one in a chain of such.
template <typename... K, typename... A>
inline wq_status launch_following(void (*kernel)(K...), unsigned grid, unsigned block, size_t smem,
                                  cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<K>(args)...) == cudaSuccess ? launch_status()
                                                                                 : WQ_ERR_CUDA;
}

// Everything before this kernel in the stream is complete and visible.
__device__ __forceinline__ void wait_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The same; then the next kernel may be set up, while this one writes. Not for a
// kernel that writes INT4 or NF4 codes, scales or zeros: the decode GEMV loads its
// weights before it waits (their kernels leave the next one's start to their end).
__device__ __forceinline__ void follow_previous() {
  wait_previous();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

inline int num_sms() {
  static int sms = [] {
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) == cudaSuccess)
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
  }();
  return sms;
}

// Allow `kernel` `bytes` of dynamic shared memory on the current device. The
// attribute belongs to a device: `done`, one per kernel, has a bit for each of
// the first 64 (later ones are set at every call).
template <typename F>
inline bool allow_smem(F kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess)
    return false;
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

// ---------------------------------------------------------------------------
// Device helpers
// ---------------------------------------------------------------------------

// 128-bit streaming load that does not allocate in L1 (read-only data).
__device__ __forceinline__ uint4 ld_stream_u4(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

__device__ __forceinline__ uint2 ld_stream_u2(const void* p) {
  uint2 r;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
               : "=r"(r.x), "=r"(r.y)
               : "l"(p));
  return r;
}

// 128-bit store with evict-first (streaming) cache policy.
__device__ __forceinline__ void st_stream_u4(void* p, uint4 v) {
  asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

// Two fp32 -> packed bf16x2 (lo in the low half), round to nearest even.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// fp32 -> bf16 bits, round to nearest even.
__device__ __forceinline__ uint16_t bf16_bits(float v) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(v));
  return r;
}

// Two fp32 -> packed fp16x2 (lo in the low half), round to nearest even.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float bf16_lo_to_f32(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi_to_f32(uint32_t v) {
  return __uint_as_float(v & 0xFFFF0000u);
}

__device__ __forceinline__ uint32_t lop3_and_or(uint32_t a, uint32_t mask, uint32_t orv) {
  // (a & mask) | orv
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(mask), "r"(orv));
  return r;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

}  // namespace wq
