// moe_activation, moe_activation_backward: the activation between an expert's two products, as calls of its own
// for a training step that keeps the first product's sums [g | u].
//
//   h  = act(g) u                      (no_mul: act(g); swigluoai: (u' + 1) g' sigmoid(1.702 g') with the clamps)
//   dg = dh act'(g) u,  du = dh act(g)  (swigluoai: 0 for what a clamp holds, the border itself passes)
//
// Bound by HBM: 6 bytes read and written a column pair forward, 10 backward (12 with h made again), some 30
// operations.  A thread takes one vector of 8 columns, its loads before their first use; each value is read and
// written once, in fp32 in between.  Vectors a thread 1 / 2 / 4 in blocks of 128 threads: SiLU of 16384 x 14336 194 / 219
// / 277 us, its gradient with h of 8192 x 14336 199 / 212 / 263; one vector in blocks of 256 196 and 199, of 512 201 and 197
// (1.41 GB each: 7.2 TB/s).
#include "moe_act.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;

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
  const long long I = (long long)p.nv * 8, v = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (v >= p.total) return;
  long long row;
  int col;
  place(p, v, row, col);
  const long long to = v * 8, at = kMul ? row * 2 * I + col : to;  // in h and dh; in gu and dgu
  float g[8], u[8], d[8], h[8], dg[8], du[8];
  load8(gu + at, g);
  if (kMul) load8(gu + at + I, u);
  if (kBackward) load8(static_cast<const T*>(p.dh) + to, d);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float slope = 0.f;
    const float a = gate<kAct, kBackward>(g[j], slope);
    float m = 1.f;  // what act(g) is multiplied by
    if (kMul) m = kAct == MOE_ACT_SWIGLUOAI ? at_least(at_most(u[j], 7.f), -7.f) + 1.f : u[j];
    h[j] = kMul ? a * m : a;
    if (kBackward) {
      dg[j] = kMul ? d[j] * slope * m : d[j] * slope;
      du[j] = kAct == MOE_ACT_SWIGLUOAI && fabsf(u[j]) > 7.f ? 0.f : d[j] * a;
    }
  }
  if (kBackward) {
    T* dgu = static_cast<T*>(p.dgu);
    store8(dgu + at, dg);
    if (kMul) store8(dgu + at + I, du);
  }
  if (!kBackward || p.h) store8(static_cast<T*>(p.h) + to, h);
}

template <class T, bool kBackward>
void launch(int act, const Act& p, cudaStream_t s) {
  const unsigned grid = (unsigned)((p.total + kThreads - 1) / kThreads);
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
  if (p.total > (1ll << 37)) return MOE_ERR_UNSUPPORTED;  // (the grid's limit; 2^40 values)
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
