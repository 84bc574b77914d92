// moe_activation, moe_activation_backward: the activation between an expert's two products, as calls of its own
// for a training step that keeps the first product's sums [g | u].
//
//   h  = act(g) u                      (no_mul: act(g); swigluoai: (u' + 1) g' sigmoid(1.702 g') with the clamps)
//   dg = dh act'(g) u,  du = dh act(g)  (swigluoai: 0 for what a clamp holds, the border itself passes)
//
// Bound by HBM: 6 bytes read and written a column pair forward, 10 backward (12 with h made again), some 30
// operations.  A thread takes two vectors of 8 columns, all loads before the first use; each value is read and
// written once, in fp32 in between.
#include "moe_act.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 2;  // vectors a thread

__device__ __forceinline__ float at_least(float z, float low) { return z < low ? low : z; }  // (a NaN stays)
__device__ __forceinline__ float at_most(float z, float high) { return z > high ? high : z; }

// act(g) and, for the gradient, act'(g).  Far below 0 the values are 0 to fp32; g kept above -128 (-16) gives that
// for -inf too, which a sum may have become in 16 bits.
template <int kAct, bool kSlope>
__device__ __forceinline__ float gate(float g, float& slope) {
  if constexpr (kAct == MOE_ACT_SWIGLUOAI) {
    const float c = at_least(at_most(g, 7.f), -128.f), q = fast_sigmoid(1.702f * c);
    if (kSlope) slope = g > 7.f ? 0.f : q * fmaf(1.702f * c, 1.0f - q, 1.0f);
    return c * q;
  } else {
    constexpr int a = kAct == MOE_ACT_GELU || kAct == MOE_ACT_GELU_NO_MUL ? MOE_LINEAR_GELU
                      : kAct == MOE_ACT_GELU_TANH                        ? MOE_LINEAR_GELU_TANH
                                                                         : MOE_LINEAR_SILU;
    if (kSlope) slope = act_grad(g, a);
    return act_fwd(at_least(g, a == MOE_LINEAR_SILU ? -128.f : -16.f), a);
  }
}

struct Act {
  const void *gu, *dh;
  void *h, *dgu;
  long long total;  // vectors of 8 columns of h
  int nv;           // of a row
};

// Row and first column of vector v.
__device__ __forceinline__ void place(const Act& p, long long v, long long& row, int& col) {
  if (p.total <= 0xFFFFFFFFll) {  // (a 64-bit division costs as much as the rest)
    const uint32_t r = (uint32_t)v / (uint32_t)p.nv;
    row = r;
    col = ((uint32_t)v - r * (uint32_t)p.nv) * 8;
  } else {
    row = v / p.nv;
    col = (int)(v - row * p.nv) * 8;
  }
}

template <class T, int kAct, bool kBackward>
__global__ void __launch_bounds__(kThreads) activation_kernel(const Act p) {
  constexpr bool kMul = kAct != MOE_ACT_SILU_NO_MUL && kAct != MOE_ACT_GELU_NO_MUL;
  const T* gu = static_cast<const T*>(p.gu);
  const long long I = (long long)p.nv * 8, v0 = (long long)blockIdx.x * (kThreads * kVecs) + threadIdx.x;
  float g[kVecs][8], u[kVecs][8], d[kVecs][8];
  long long at[kVecs], to[kVecs];  // in gu and dgu; in h and dh
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const long long v = v0 + i * kThreads;
    if (v >= p.total) continue;
    long long row;
    int col;
    place(p, v, row, col);
    to[i] = v * 8;
    at[i] = kMul ? row * 2 * I + col : to[i];
    load8(gu + at[i], g[i]);
    if (kMul) load8(gu + at[i] + I, u[i]);
    if (kBackward) load8(static_cast<const T*>(p.dh) + to[i], d[i]);
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    if (v0 + i * kThreads >= p.total) continue;
    float h[8], dg[8], du[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float slope = 0.f;
      const float a = gate<kAct, kBackward>(g[i][j], slope);
      float m = 1.f;  // what act(g) is multiplied by
      if (kMul) m = kAct == MOE_ACT_SWIGLUOAI ? at_least(at_most(u[i][j], 7.f), -7.f) + 1.f : u[i][j];
      h[j] = kMul ? a * m : a;
      if (kBackward) {
        dg[j] = kMul ? d[i][j] * slope * m : d[i][j] * slope;
        du[j] = kAct == MOE_ACT_SWIGLUOAI && fabsf(u[i][j]) > 7.f ? 0.f : d[i][j] * a;
      }
    }
    if (kBackward) {
      T* dgu = static_cast<T*>(p.dgu);
      store8(dgu + at[i], dg);
      if (kMul) store8(dgu + at[i] + I, du);
    }
    if (!kBackward || p.h) store8(static_cast<T*>(p.h) + to[i], h);
  }
}

template <class T, bool kBackward>
void launch(int act, const Act& p, cudaStream_t s) {
  const long long per = kThreads * kVecs;
  const unsigned grid = (unsigned)((p.total + per - 1) / per);
  switch (act) {
    case MOE_ACT_SILU: activation_kernel<T, MOE_ACT_SILU, kBackward><<<grid, kThreads, 0, s>>>(p); break;
    case MOE_ACT_GELU: activation_kernel<T, MOE_ACT_GELU, kBackward><<<grid, kThreads, 0, s>>>(p); break;
    case MOE_ACT_GELU_TANH: activation_kernel<T, MOE_ACT_GELU_TANH, kBackward><<<grid, kThreads, 0, s>>>(p); break;
    case MOE_ACT_SWIGLUOAI: activation_kernel<T, MOE_ACT_SWIGLUOAI, kBackward><<<grid, kThreads, 0, s>>>(p); break;
    case MOE_ACT_SILU_NO_MUL: activation_kernel<T, MOE_ACT_SILU_NO_MUL, kBackward><<<grid, kThreads, 0, s>>>(p); break;
    default: activation_kernel<T, MOE_ACT_GELU_NO_MUL, kBackward><<<grid, kThreads, 0, s>>>(p);
  }
}

template <bool kBackward>
moe_status_t run(const void* dh, const void* gu, int S, int I, moe_dtype_t dtype, int act, void* dgu, void* h,
                 moe_stream_t stream) {
  MOE_CHECK_ARG(S >= 0 && S <= (1 << 30) && I >= 8 && I % 8 == 0 && I <= (1 << 21));
  if (dtype != MOE_DT_BF16 && dtype != MOE_DT_FP16) return MOE_ERR_UNSUPPORTED;
  if (act < MOE_ACT_SILU || act > MOE_ACT_GELU_NO_MUL) return MOE_ERR_UNSUPPORTED;
  if (S == 0) return MOE_OK;
  MOE_CHECK_ARG(gu && (kBackward ? dh && dgu : h != nullptr));
  MOE_CHECK_ARG(aligned16(gu) && aligned16(dh) && aligned16(dgu) && aligned16(h));
  const Act p{gu, dh, h, dgu, (long long)S * (I / 8), I / 8};
  if (p.total > (1ll << 39)) return MOE_ERR_UNSUPPORTED;  // (the grid's limit; 2^42 values)
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == MOE_DT_FP16)
    launch<__half, kBackward>(act, p, s);
  else
    launch<__nv_bfloat16, kBackward>(act, p, s);
  return launch_status();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_activation(const void* gu, int S, int I, moe_dtype_t dtype, int activation, void* h,
                                       moe_stream_t stream) {
  return run<false>(nullptr, gu, S, I, dtype, activation, nullptr, h, stream);
}

extern "C" moe_status_t moe_activation_backward(const void* dh, const void* gu, int S, int I, moe_dtype_t dtype,
                                                int activation, void* dgu, void* h, moe_stream_t stream) {
  return run<true>(dh, gu, S, I, dtype, activation, dgu, h, stream);
}
