// Shared by the training operators (moeskew_train.h): launchers, 8- and 4-element loads and
// stores in fp32 from either element type, and launches that overlap their predecessor.
#pragma once

#include <cuda_bf16.h>

#include "moe_common.cuh"
#include "moeskew_train.h"

namespace moe {

// ---- launchers, called by the C ABI after validation ----
size_t balance_workspace_bytes(const moe_cfg& c, int n_seq);
cudaError_t launch_balance_loss(const moe_cfg& c, const float* logits, const int32_t* ids,
                                const uint8_t* mask, const int32_t* seq_off, int n_seq,
                                float* losses, int32_t* counts, float* probs,
                                int32_t* seq_info, float* lse, void* ws, int32_t* status,
                                cudaStream_t st);
cudaError_t launch_router_backward(const moe_cfg& c, const float* logits, const int32_t* ids,
                                   const float* gates, const float* dy, const uint16_t* o,
                                   const int32_t* tok_row, const uint8_t* mask,
                                   const int32_t* seq_off, int n_seq, const int32_t* counts,
                                   const int32_t* seq_info, const float* lse,
                                   const float* dloss, float* dgates, float* dlogits,
                                   int32_t* status, cudaStream_t st);
size_t norm_bwd_workspace_bytes(const moe_cfg& c);
cudaError_t launch_block_norm(const moe_cfg& c, const moet_norm& n, const void* h,
                              const float* y, const float* gate, const void* w_post,
                              const void* w_next, void* h_out, uint16_t* x, cudaStream_t st);
cudaError_t launch_block_norm_backward(const moe_cfg& c, const moet_norm& n,
                                       const void* h_out, const float* y, const float* gate,
                                       const void* w_post, const void* w_next,
                                       const void* dh_out, const float* dx, void* dh,
                                       float* dy, float* dgate, float* dw_post,
                                       float* dw_next, void* ws, cudaStream_t st);
cudaError_t launch_adamw(const moet_adamw_tensor* tensors, int count, const moet_adamw& opt,
                         const float* lr, const float* grad_scale, int32_t* step,
                         cudaStream_t st);

// ---- element access ----
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[0];
  const float4 b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void bf16x8_to_f32(const uint4 a, float* v) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// ---- copies ahead of time, 16 (or 8) bytes from global to shared memory, read back by the
// thread that made them after wait_copies() (so no barrier guards them) ----
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void copy_ahead16(uint32_t dst, const void* src) {
  // through L1: the second half of a 32-byte sector that two copies share hits there
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_ahead8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void commit_copies() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int LEFT>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}
__device__ __forceinline__ uint4 slot16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Sums of N = 2, 4 or 8 values over the warp, of 8 with 9 shuffles: each of the first log2 N
// exchanges halves the number of values a lane still carries.  Lane l returns the sum of value
// l / (32 / N).
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N], int lane) {
#pragma unroll
  for (int half = N / 2, off = 16; half >= 1; half >>= 1, off >>= 1) {
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
    }
  }
#pragma unroll
  for (int off = 16 / N; off >= 1; off >>= 1)
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
  return v[0];
}

// ---- launches that overlap their predecessor's end (programmatic dependent launch) ----
// The dependent kernel calls wait_for_predecessor() before it touches what the kernels
// before it wrote; that returns once the predecessor has ended and its writes are visible.
__device__ __forceinline__ void wait_for_predecessor() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_successor_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <class... KArgs, class... Args>
cudaError_t launch_after(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                         cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

}  // namespace moe
