// moe_finalize_backward: gradients of the finalize (weighted sum of the top-k rows, shared
// row and residual, then the optional RMSNorm).
//
//   G = r (gamma dn - o r^2 mean(gamma dn o)) + dres,   r = 1 / sqrt(mean(o^2) + eps)
//   dy_j = w_j G,  dw_j = <G, y_j>,  dsum = G,  drms = sum_t dn o r
//
// Bound by HBM: a token moves 2 H (4 + 2 top_k) bytes and computes a few operations per
// element.  A CTA takes whole tokens, G stays in registers between the norm's two sums and the
// top_k rows, and each element is read once.  drms: every thread owns the same columns for all
// tokens of its CTA and adds them in shared memory; one row of partial sums per CTA goes to the
// workspace and a second launch adds the rows in order (a fixed order: the same bits each time).
#include "moe_vec.cuh"

namespace moe {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxK = 32;

struct FinBwd {
  const __nv_bfloat16 *dout, *dres, *o, *gamma, *y;
  const float* w;
  float eps;
  int T, H, k;
  __nv_bfloat16 *dy, *dsum;
  float *dw, *partial;
};

// NV: 8-element vectors of a row held by a thread.
template <int NV>
__global__ void __launch_bounds__(kMaxThreads)
    finalize_backward_kernel(const FinBwd a) {
  extern __shared__ __align__(16) float drms_sum[];  // [H] when partial
  __shared__ float red[2][kMaxThreads / 32];
  __shared__ float dots[kMaxK][kMaxThreads / 32];
  const int nvec = a.H / 8, warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (a.partial)
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) drms_sum[i] = 0.f;
  __syncthreads();
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    float g[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nvec) load8(a.dout + (size_t)t * a.H + v * 8, g[i]);
    }
    if (a.gamma) {
      float o[NV][8], sq = 0.f, gd = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= nvec) continue;
        float gm[8];
        load8(a.o + (size_t)t * a.H + v * 8, o[i]);
        load8(a.gamma + v * 8, gm);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sq += o[i][e] * o[i][e];
          gd += g[i][e] * gm[e] * o[i][e];
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        sq += __shfl_xor_sync(0xffffffffu, sq, off);
        gd += __shfl_xor_sync(0xffffffffu, gd, off);
      }
      if (lane == 0) {
        red[0][warp] = sq;
        red[1][warp] = gd;
      }
      __syncthreads();
      sq = gd = 0.f;
      for (int i = 0; i < warps; ++i) {
        sq += red[0][i];
        gd += red[1][i];
      }
      const float r = __frsqrt_rn(sq / a.H + a.eps);
      const float c = r * r * (gd / a.H);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= nvec) continue;
        float gm[8];
        load8(a.gamma + v * 8, gm);
        if (a.partial) {
#pragma unroll
          for (int e = 0; e < 8; ++e) drms_sum[v * 8 + e] += g[i][e] * o[i][e] * r;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) g[i][e] = r * (g[i][e] * gm[e] - o[i][e] * c);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec) continue;
      if (a.dres) {
        float d[8];
        load8(a.dres + (size_t)t * a.H + v * 8, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[i][e] += d[e];
      }
      if (a.dsum) store8(a.dsum + (size_t)t * a.H + v * 8, g[i]);
    }
    for (int j = 0; j < a.k; ++j) {
      const size_t row = ((size_t)t * a.k + j) * a.H;
      const float w = a.w ? __ldg(a.w + (size_t)t * a.k + j) : 1.f;
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= nvec) continue;
        if (a.dw) {
          float y[8];
          load8(a.y + row + v * 8, y);
#pragma unroll
          for (int e = 0; e < 8; ++e) dot += g[i][e] * y[e];
        }
        if (a.dy) {
          float d[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] = w * g[i][e];
          store8(a.dy + row + v * 8, d);
        }
      }
      if (a.dw) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        if (lane == 0) dots[j][warp] = dot;
      }
    }
    __syncthreads();
    if (a.dw && threadIdx.x < a.k) {
      float s = 0.f;
      for (int i = 0; i < warps; ++i) s += dots[threadIdx.x][i];
      a.dw[(size_t)t * a.k + threadIdx.x] = s;
    }
    __syncthreads();
  }
  if (a.partial)
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) a.partial[(size_t)blockIdx.x * a.H + i] = drms_sum[i];
}

// out[h] = sum over p of partial[p][h], p in ascending order within each of 8 interleaved sums.
__global__ void __launch_bounds__(256) drms_kernel(const float* __restrict__ partial, int P, int H, float* out) {
  __shared__ float sums[8][32];
  const int h = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  float s = 0.f;
  if (h < H)
    for (int p = part; p < P; p += 8) s += partial[(size_t)p * H + h];
  sums[part][threadIdx.x & 31] = s;
  __syncthreads();
  if (part == 0 && h < H) {
    for (int i = 1; i < 8; ++i) s += sums[i][threadIdx.x & 31];
    out[h] = s;
  }
}

constexpr int kMaxH = 16384;

// Threads a token and vectors a thread: the fewest vectors (up to 4) that keep a row within
// kMaxThreads threads.
void shape(int H, int* threads, int* nv) {
  const int nvec = H / 8;
  *nv = nvec <= 256 ? 1 : nvec <= 512 ? 2 : 4;
  *threads = ((nvec + *nv - 1) / *nv + 31) / 32 * 32;
}

int grid_ctas(int T) { return (int)((long long)T < 4LL * num_sms() ? T : 4LL * num_sms()); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_finalize_backward_workspace_size(int T, int H) {
  if (T <= 0 || H <= 0) return 0;
  return (size_t)grid_ctas(T) * (size_t)H * sizeof(float);
}

extern "C" moe_status_t moe_finalize_backward(const void* dout, const void* dresidual_out, const void* residual_out,
                                              const void* rms_weight, float eps, const void* fused_expert_output,
                                              const float* topk_weights, int T, int H, int top_k, void* dy,
                                              float* dweights, void* dsum, float* drms, void* ws, size_t ws_bytes,
                                              moe_stream_t stream) {
  MOE_CHECK_ARG(T >= 0 && H > 0 && H % 8 == 0 && top_k >= 1 && top_k <= kMaxK && eps >= 0.f);
  MOE_CHECK_ARG(dy || dweights || dsum || drms);
  MOE_CHECK_ARG(!drms || rms_weight);
  if (H > kMaxH) return MOE_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  MOE_CHECK_ARG(aligned16(drms));
  if (T == 0) {
    if (drms && cudaMemsetAsync(drms, 0, (size_t)H * sizeof(float), s) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  MOE_CHECK_ARG(dout && (!rms_weight || residual_out) && (!dweights || (topk_weights && fused_expert_output)));
  MOE_CHECK_ARG(aligned16(dout) && aligned16(dresidual_out) && aligned16(residual_out) && aligned16(rms_weight) &&
                aligned16(fused_expert_output) && aligned16(topk_weights) && aligned16(dy) && aligned16(dweights) &&
                aligned16(dsum) && aligned16(ws));
  if (drms && (!ws || ws_bytes < moe_finalize_backward_workspace_size(T, H))) return MOE_ERR_WORKSPACE;
  FinBwd a;
  a.dout = static_cast<const __nv_bfloat16*>(dout);
  a.dres = static_cast<const __nv_bfloat16*>(dresidual_out);
  a.o = static_cast<const __nv_bfloat16*>(residual_out);
  a.gamma = static_cast<const __nv_bfloat16*>(rms_weight);
  a.y = static_cast<const __nv_bfloat16*>(fused_expert_output);
  a.w = topk_weights;
  a.eps = eps;
  a.T = T;
  a.H = H;
  a.k = top_k;
  a.dy = static_cast<__nv_bfloat16*>(dy);
  a.dsum = static_cast<__nv_bfloat16*>(dsum);
  a.dw = dweights;
  a.partial = drms ? static_cast<float*>(ws) : nullptr;
  int threads, nv;
  shape(H, &threads, &nv);
  const int grid = grid_ctas(T);
  const size_t smem = drms ? (size_t)H * sizeof(float) : 0;
  auto run = [&](auto kern) {
    if (smem > 40 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kMaxH * sizeof(float))) != cudaSuccess)
      return false;
    kern<<<grid, threads, smem, s>>>(a);
    return true;
  };
  const bool ok = nv == 1 ? run(finalize_backward_kernel<1>)
                          : nv == 2 ? run(finalize_backward_kernel<2>) : run(finalize_backward_kernel<4>);
  if (!ok) return MOE_ERR_CUDA;
  if (drms) drms_kernel<<<(H + 31) / 32, 256, 0, s>>>(a.partial, grid, H, drms);
  return launch_status();
}
