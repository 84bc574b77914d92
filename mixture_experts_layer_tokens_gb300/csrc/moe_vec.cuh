// Typed element and vector access of the linear, grouped-route and gradient kernels: fp32,
// bf16 and fp16 values in and out of fp32 registers.
#pragma once
#include <cuda_fp16.h>

#include <type_traits>

#include "moe_common.cuh"

namespace moe {

moe_status_t route_grouped_status(int clear);
moe_status_t linear_status(int clear);
moe_status_t grouped_status(int clear);
moe_status_t rmsnorm_status(int clear);
moe_status_t finalize_backward_status(int clear);

// ---- launches that overlap the end of the launch before them on the stream
// A call's second and later kernels are launched with overlap_attr(): the device may start their
// CTAs when every CTA of the kernel before has called depend_launch() (or ended) and there is room
// for them.  depend_wait() then waits until that kernel has ended and its writes are visible.  Each
// kernel of a call waits before it touches what another kernel of the call writes, or writes what
// another one reads, and in any case before it ends, so the whole chain is ordered.  The first
// kernel of a call is launched plainly and waits for nothing; so the caller's own inputs (weights,
// offsets, slots) are complete, and outputs that this kernel alone touches are free, for every kernel of
// the call without a wait.
__device__ __forceinline__ void depend_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void depend_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

inline cudaLaunchAttribute overlap_attr() {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}
template <class... P, class... A>
cudaError_t launch_overlapped(void (*kern)(P...), int grid, int block, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {overlap_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// exp(x) and 1 / x by the special-function unit: within (2 + 1.2 |x|) 2^-23 (the product with
// log2 e rounds) and 1 ulp; results below 2^-126 are 0.
__device__ __forceinline__ float fast_exp(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
  return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float load1(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }
__device__ __forceinline__ float load1(const __half* p) { return __half2float(__ldg(p)); }

__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(__half* p, float v) { *p = __float2half_rn(v); }

// 4 bytes of packed values <-> fp32
template <class T>
struct Word;
template <>
struct Word<float> {
  static constexpr int N = 1;
  static __device__ __forceinline__ void get(uint32_t w, float* v) { v[0] = __uint_as_float(w); }
  static __device__ __forceinline__ uint32_t put(const float* v) { return __float_as_uint(v[0]); }
};
template <>
struct Word<__nv_bfloat16> {
  static constexpr int N = 2;
  static __device__ __forceinline__ void get(uint32_t w, float* v) {
    v[0] = bf16lo(w);
    v[1] = bf16hi(w);
  }
  static __device__ __forceinline__ uint32_t put(const float* v) { return pack_bf16x2(v[0], v[1]); }
};
template <>
struct Word<__half> {
  static constexpr int N = 2;
  static __device__ __forceinline__ void get(uint32_t w, float* v) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    v[0] = f.x;
    v[1] = f.y;
  }
  static __device__ __forceinline__ uint32_t put(const float* v) {
    const __half2 h = __floats2half2_rn(v[0], v[1]);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// 8 consecutive values (16-byte aligned) <-> fp32
template <class T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  constexpr int W = 8 / Word<T>::N;  // words
  uint32_t w[W];
#pragma unroll
  for (int i = 0; i < W; i += 4) {
    const uint4 q = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
    w[i] = q.x;
    w[i + 1] = q.y;
    w[i + 2] = q.z;
    w[i + 3] = q.w;
  }
#pragma unroll
  for (int i = 0; i < W; ++i) Word<T>::get(w[i], v + i * Word<T>::N);
}
template <class T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  constexpr int W = 8 / Word<T>::N;
  uint32_t w[W];
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = Word<T>::put(v + i * Word<T>::N);
#pragma unroll
  for (int i = 0; i < W; i += 4)
    *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(p) + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
}

// NV consecutive elements at p, of which the first cnt exist (-inf for the rest); by vectors of
// up to 16 bytes when they tile `period`, the distance that p's offset and cnt are made of.
template <int NV, class T>
__device__ __forceinline__ void load_lane(const T* p, int cnt, int period, float (&v)[NV]) {
  constexpr int BYTES = NV * (int)sizeof(T) < 16 ? NV * (int)sizeof(T) : 16;
  constexpr int PER = BYTES / (int)sizeof(T);  // elements of a vector
  if constexpr (BYTES >= 4) {
    if (period % PER == 0) {
#pragma unroll
      for (int i = 0; i < NV; i += PER) {
        if (i < cnt) {
          uint32_t w[BYTES / 4];
          if constexpr (BYTES == 16) {
            const uint4 q = __ldg(reinterpret_cast<const uint4*>(p + i));
            w[0] = q.x;
            w[1] = q.y;
            w[2] = q.z;
            w[3] = q.w;
          } else if constexpr (BYTES == 8) {
            const uint2 q = __ldg(reinterpret_cast<const uint2*>(p + i));
            w[0] = q.x;
            w[1] = q.y;
          } else {
            w[0] = __ldg(reinterpret_cast<const uint32_t*>(p + i));
          }
#pragma unroll
          for (int j = 0; j < BYTES / 4; ++j) Word<T>::get(w[j], v + i + j * Word<T>::N);
        } else {
#pragma unroll
          for (int j = 0; j < PER; ++j) v[i + j] = -INFINITY;
        }
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = i < cnt ? load1(p + i) : -INFINITY;
}

// A row of n fp32 values in shared memory (16-byte aligned) written by one warp as type T.
template <class T>
__device__ __forceinline__ void store_row(T* row, int n, int lane, const float* buf) {
  constexpr int PER = 16 / (int)sizeof(T);
  if (n % PER == 0) {
    for (int i = lane * PER; i < n; i += 32 * PER) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = Word<T>::put(buf + i + j * Word<T>::N);
      *reinterpret_cast<uint4*>(row + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    for (int i = lane; i < n; i += 32) store1(row + i, buf[i]);
  }
}

}  // namespace moe
