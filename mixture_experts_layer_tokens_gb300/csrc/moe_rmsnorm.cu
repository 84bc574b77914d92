// moe_rmsnorm: RMSNorm in front of the layer, with the residual's addition before it and the 8-bit rows that the fp8
// experts take behind it, in one pass.
//
//   v = x + residual;  residual_out = bf16(v);  n = v gamma / sqrt(mean(v^2) + eps);  out = bf16(n)
//   s = max(max |n|, 1e-10) / 448 over 128 columns or the row;  q = e4m3(n / s)
//
// Bound by HBM: up to 9 bytes a value (x, residual, residual_out, out, q) and a dozen operations.  A group of
// threads takes a row and keeps it in registers between the sum of squares and the outputs, so each value is read
// and written once; the 16 lanes whose vectors make 128 columns find their scale by shuffles.
#include "moe_vec.cuh"

namespace moe {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxH = 16384;

struct Norm {
  const __nv_bfloat16 *x, *res, *gamma;
  __nv_bfloat16 *out, *res_out;
  uint8_t* q;
  float* scale;
  float eps;
  int T, H;
  int group;    // 0 (no q), 128 or MOE_GROUP_TOKEN
  int threads;  // of a row: 16 or a multiple of 32
};

// Over the `threads` lanes of a row (16, or whole warps); the same value in each.
template <bool kMax>
__device__ __forceinline__ float row_reduce(float a, int threads, float (&red)[2][kMaxThreads / 32], int which) {
  auto op = [](float p, float q) { return kMax ? fmaxf(p, q) : p + q; };
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) a = op(a, __shfl_xor_sync(0xffffffffu, a, off));
  if (threads == 16) return a;
  a = op(a, __shfl_xor_sync(0xffffffffu, a, 16));
  const int warps = threads >> 5;
  if (warps == 1) return a;
  const int warp = threadIdx.x >> 5, first = warp / warps * warps;
  if ((threadIdx.x & 31) == 0) red[which][warp] = a;
  __syncthreads();
  a = red[which][first];
  for (int i = 1; i < warps; ++i) a = op(a, red[which][first + i]);
  return a;
}

// NV: vectors of 8 columns a thread holds of a row.
template <int NV>
__global__ void rmsnorm_kernel(const Norm p) {
  __shared__ float red[2][kMaxThreads / 32];
  const int threads = p.threads, rows = blockDim.x / threads;  // rows of a CTA at a time
  const int i = threadIdx.x % threads, nvec = p.H / 8;
  float gamma[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = j * threads + i;
    if (v < nvec) load8(p.gamma + v * 8, gamma[j]);
  }
  // (every thread of the CTA makes every turn: the sums meet at barriers)
  for (int t0 = blockIdx.x * rows; t0 < p.T; t0 += gridDim.x * rows) {
    const int t = t0 + threadIdx.x / threads;
    const size_t at = (size_t)t * p.H;
    float n[NV][8], sum = 0.f;
    bool on[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = j * threads + i;
      on[j] = t < p.T && v < nvec;
      if (on[j]) {
        load8(p.x + at + v * 8, n[j]);
        if (p.res) {
          float r[8];
          load8(p.res + at + v * 8, r);
#pragma unroll
          for (int c = 0; c < 8; ++c) n[j][c] += r[c];
        }
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) n[j][c] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int c = 0; c < 8; ++c) sum = fmaf(n[j][c], n[j][c], sum);
    if (p.res_out) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on[j]) store8(p.res_out + at + (size_t)(j * threads + i) * 8, n[j]);
    }
    const float r = __frsqrt_rn(row_reduce<false>(sum, threads, red, 0) / (float)p.H + p.eps);
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (on[j]) {
#pragma unroll
        for (int c = 0; c < 8; ++c) n[j][c] = n[j][c] * r * gamma[j][c];
        if (p.out) store8(p.out + at + (size_t)(j * threads + i) * 8, n[j]);
      }
    }
    if (p.group == MOE_GROUP_TOKEN) {
#pragma unroll
      for (int j = 0; j < NV; ++j) most = fmaxf(most, amax8(n[j]));
      const float s = __fdiv_rn(fmaxf(row_reduce<true>(most, threads, red, 1), 1e-10f), 448.f);
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on[j]) *reinterpret_cast<uint2*>(p.q + at + (size_t)(j * threads + i) * 8) = e4m3x8(n[j], s);
      if (i == 0 && t < p.T) p.scale[t] = s;
    } else if (p.group) {
      const int groups = (p.H + 127) / 128;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float a = amax8(n[j]);
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
        const float s = __fdiv_rn(fmaxf(a, 1e-10f), 448.f);
        const int v = j * threads + i;
        if (on[j]) {
          *reinterpret_cast<uint2*>(p.q + at + (size_t)v * 8) = e4m3x8(n[j], s);
          if (v % 16 == 0) p.scale[(size_t)t * groups + v / 16] = s;
        }
      }
    }
    __syncthreads();  // (red is written again)
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_rmsnorm(const void* x, const void* residual, const void* weight, float eps, int T, int H,
                                    const moe_quant_config* qc, void* out, void* residual_out, void* q, float* q_scale,
                                    moe_stream_t stream) {
  MOE_CHECK_ARG(T >= 0 && T <= (1 << 30) && H >= 8 && H % 8 == 0 && H <= kMaxH);
  MOE_CHECK_ARG(eps >= 0.f && eps <= 3e38f);
  int group = 0;
  if (qc && qc->act != MOE_DT_BF16) {
    if (qc->act != MOE_DT_FP8_E4M3 || (qc->act_group != 128 && qc->act_group != MOE_GROUP_TOKEN))
      return MOE_ERR_UNSUPPORTED;
    group = qc->act_group;
  }
  if (T == 0) return MOE_OK;
  MOE_CHECK_ARG(x && weight && (out || group) && (group ? q && q_scale : !q && !q_scale));
  MOE_CHECK_ARG(aligned16(x) && aligned16(residual) && aligned16(weight) && aligned16(out) && aligned16(residual_out) &&
                aligned16(q) && aligned16(q_scale));
  using B = __nv_bfloat16;
  Norm p{static_cast<const B*>(x), static_cast<const B*>(residual), static_cast<const B*>(weight), static_cast<B*>(out),
         static_cast<B*>(residual_out), static_cast<uint8_t*>(q), q_scale, eps, T, H, group, 0};
  const int nvec = H / 8;
  auto go = [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    const int need = (nvec + NV - 1) / NV;
    p.threads = need <= 16 ? 16 : (need + 31) / 32 * 32;
    const int rows = p.threads >= 128 ? 1 : 128 / p.threads, block = rows * p.threads;
    const int turns = (T + rows - 1) / rows, most = num_sms() * (2048 / block);
    rmsnorm_kernel<NV><<<turns < most ? turns : most, block, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  };
  // a row's loads in one round where there are few rows, fewer threads to a row where there are many
  if (nvec <= kMaxThreads && T <= num_sms())
    go(std::integral_constant<int, 1>());
  else
    go(std::integral_constant<int, 4>());
  return launch_status();
}
