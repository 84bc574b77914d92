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
constexpr int kRegs = 65536;  // of an SM
constexpr int kMaxSmem = 2 * 2 * kMaxH * 2;  // two stages of two rows
// A sum of squares below 2^-80 has lost digits to those that vanish in fp32 (each is off by up to 2^-150, by 2^-136 in
// all), which counts where eps is no larger: such a row is multiplied by 2^100, exactly, and summed again.  (A kernel of
// its own: the branch cost the others 1.3 %, 16384 x 7168 162.8 -> 165.0 us.)
constexpr float kSmall = 0x1p-80f, kRaise = 0x1p100f;

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

// Over the `threads` lanes of a row (16, or whole warps); the same value in each.  Every thread of the CTA comes.
template <bool kMax>
__device__ __forceinline__ float row_reduce(float a, int threads, float* red) {
  auto op = [](float p, float q) { return kMax ? fmaxf(p, q) : p + q; };
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) a = op(a, __shfl_xor_sync(0xffffffffu, a, off));
  if (threads > 16) a = op(a, __shfl_xor_sync(0xffffffffu, a, 16));
  const int warp = threadIdx.x >> 5, warps = threads >> 5;
  if (warps > 1 && (threadIdx.x & 31) == 0) red[warp] = a;
  __syncthreads();
  if (warps > 1) {
    const int first = warp / warps * warps;
    a = red[first];
    for (int i = 1; i < warps; ++i) a = op(a, red[first + i]);
  }
  return a;
}

__device__ __forceinline__ void unpack8(const uint4 w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) Word<__nv_bfloat16>::get(u[i], v + 2 * i);
}

__device__ __forceinline__ void bulk_load(void* smem_dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(smem_dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// NV: vectors of 8 columns a thread holds of a row.  kRing: the rows come through two stages of shared memory by bulk
// copies, the next turn's under this turn's work (loads by the threads themselves left HBM idle through each row's
// sum and outputs: 16384 x 7168 with all outputs 301 us).  kSmallEps: eps is below kSmall.
template <int NV, bool kRing, bool kSmallEps>
__global__ void __launch_bounds__(NV == 4 ? kMaxThreads / 2 : kMaxThreads) rmsnorm_kernel(const Norm p) {
  extern __shared__ __align__(128) uint8_t stages[];
  __shared__ float red[kSmallEps ? 3 : 2][2][kMaxThreads / 32];
  __shared__ uint64_t full[2];
  const int threads = p.threads, rows = blockDim.x / threads;  // rows of a CTA at a time
  const int i = threadIdx.x % threads, mine = threadIdx.x / threads, nvec = p.H / 8;
  const size_t tensor = (size_t)rows * p.H * 2;  // bytes of one tensor's rows in a stage
  const int step = gridDim.x * rows;
  bool ok = true;
  auto fetch = [&](int t0, int stage) {  // by one thread
    if (t0 >= p.T) return;
    const uint32_t bytes = (uint32_t)min(rows, p.T - t0) * p.H * 2;
    uint8_t* to = stages + stage * tensor * (p.res ? 2 : 1);
    mbar_arrive_expect_tx(&full[stage], p.res ? 2 * bytes : bytes);
    bulk_load(to, p.x + (size_t)t0 * p.H, bytes, &full[stage]);
    if (p.res) bulk_load(to + tensor, p.res + (size_t)t0 * p.H, bytes, &full[stage]);
  };
  if (kRing) {
    if (threadIdx.x == 0) {
      mbar_init(&full[0], 1);
      mbar_init(&full[1], 1);
      fence_mbar_init();
      fetch(blockIdx.x * rows, 0);
      fetch(blockIdx.x * rows + step, 1);
    }
    __syncthreads();
  }
  uint4 gamma[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = j * threads + i;
    if (v < nvec) gamma[j] = __ldg(reinterpret_cast<const uint4*>(p.gamma) + v);
  }
  // (every thread of the CTA makes every turn: the sums meet at barriers)
  int turn = 0;
  for (int t0 = blockIdx.x * rows; t0 < p.T; t0 += step, ++turn) {
    const int t = t0 + mine, stage = turn & 1;
    const size_t at = (size_t)t * p.H;
    float n[NV][8], sum = 0.f;
    bool on[NV];
    // a wait that gives up (recorded) leaves wrong values, but every barrier is still met
    if (kRing) ok &= mbar_wait(&full[stage], turn >> 1 & 1);
    const uint8_t* row = stages + stage * tensor * (p.res ? 2 : 1) + (size_t)mine * p.H * 2;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = j * threads + i;
      on[j] = t < p.T && v < nvec;
      if (on[j]) {
        const uint4 a = kRing ? *reinterpret_cast<const uint4*>(row + v * 16)
                              : *reinterpret_cast<const uint4*>(p.x + at + v * 8);
        unpack8(a, n[j]);
        if (p.res) {
          const uint4 b = kRing ? *reinterpret_cast<const uint4*>(row + tensor + v * 16)
                                : *reinterpret_cast<const uint4*>(p.res + at + v * 8);
          float r[8];
          unpack8(b, r);
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
    sum = row_reduce<false>(sum, threads, red[0][stage]);
    if (kRing && threadIdx.x == 0) fetch(t0 + 2 * step, stage);  // (all threads have read the stage)
    if (p.res_out) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on[j]) store8(p.res_out + at + (size_t)(j * threads + i) * 8, n[j]);
    }
    float eps = p.eps;
    if constexpr (kSmallEps) {
      const float raise = sum < kSmall ? kRaise : 1.f;
      eps = eps * raise * raise;
      sum = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          n[j][c] *= raise;
          sum = fmaf(n[j][c], n[j][c], sum);
        }
      sum = row_reduce<false>(sum, threads, red[2][stage]);
    }
    const float r = __frsqrt_rn(sum / (float)p.H + eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (on[j]) {
        float g[8];
        unpack8(gamma[j], g);
#pragma unroll
        for (int c = 0; c < 8; ++c) n[j][c] = n[j][c] * r * g[c];
        if (p.out) store8(p.out + at + (size_t)(j * threads + i) * 8, n[j]);
      }
    }
    if (p.group == MOE_GROUP_TOKEN) {
      float most = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) most = fmaxf(most, amax8(n[j]));
      const float s = __fdiv_rn(fmaxf(row_reduce<true>(most, threads, red[1][stage]), 1e-10f), 448.f);
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
  }
  // copies that a wait did not see land (bounded) before the shared memory goes
  if (kRing && !ok && threadIdx.x == 0)
    for (int s = 0; s < 2; ++s) {
      const int last = turn - 1 - ((turn - 1 - s) & 1);  // the stage's last turn
      if (last >= 0) mbar_wait(&full[s], last >> 1 & 1, false, 100000000ull);
    }
}

}  // namespace

MOE_DEFINE_STATUS_READER(rmsnorm_status)

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
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int nvec = H / 8;
  auto go = [&](auto nv, auto ring, auto small_eps) {
    constexpr int NV = decltype(nv)::value;
    constexpr bool kRing = decltype(ring)::value;
    constexpr auto kernel = rmsnorm_kernel<NV, kRing, decltype(small_eps)::value>;
    const int need = (nvec + NV - 1) / NV;
    p.threads = need <= 16 ? 16 : (need + 31) / 32 * 32;
    int rows = p.threads >= 128 ? 1 : 128 / p.threads;
    if (NV == 4)
      while (2 * rows * p.threads <= 512 && (long long)2 * rows * num_sms() <= T) rows *= 2;
    const int block = rows * p.threads;
    const int turns = (T + rows - 1) / rows;
    const int smem = kRing ? 2 * rows * H * 2 * (residual ? 2 : 1) : 0;
    int ctas = 2048 / block;  // of an SM
    if (kRing) {
      const int by_regs = kRegs / (block * (NV == 4 ? 104 : 64)), by_smem = 232448 / (smem + 2048);
      ctas = by_regs < by_smem ? by_regs : by_smem;
      if (ctas < 1) ctas = 1;
      // (the same for every call: host threads may come at once)
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess)
        return MOE_ERR_CUDA;
    }
    const int most = num_sms() * ctas;
    kernel<<<turns < most ? turns : most, block, smem, s>>>(p);
    return launch_status();
  };
  if (eps < kSmall) return go(std::integral_constant<int, 2>(), std::true_type(), std::true_type());
  // Few rows: one round of loads a thread and no ring.  All outputs, so / by the ring, us in a graph: [1, 2048] 2.3 / 2.6,
  // [150, 2048] 2.7 / 3.1, [150, 256] 2.3 / 2.8, [1, 7168] 3.3 either way, [100, 7168] 3.7 / 3.6.
  if (nvec <= kMaxThreads && T <= num_sms()) return go(std::integral_constant<int, 1>(), std::false_type(), std::false_type());
  // Many long rows: four vectors a thread and one CTA of up to 512 threads an SM, whose copies are long and neighbours in
  // memory; else two vectors, and CTAs of one row or 128 threads.  All outputs, two vectors / four in CTAs of one row or
  // 128 threads / four in CTAs of 512: [16384, 7168] 185 / 179 / 162 us, [16384, 2048] 57 / 55 / 49, [16384, 1024] 29 / 28 /
  // 27, [16384, 256] 9.0 / 12 / 12, [65536, 128] 15 / 24 / 25, [1024, 7168] 13.4 / 15 / 16 (by the threads' own loads 300,
  // 76, 39, 15, 32, 23).  Around the cut, two / four in CTAs of 512: [2048, 512] 3.4 / 3.8, [2048, 7168] 22.7 / 25.5,
  // [4096, 2048] 13.0 / 16.5, [4096, 7168] 47.6 / 46.0, [6000, 512] 5.6 / 7.9, [8192, 2048] 26.7 / 27.4, [8192, 7168] 94 / 84,
  // [12000, 2048] 41.4 / 36.6: four pay from some 2^24 values on, and cost up to 40 % between the cut and there.
  if (nvec >= 64 && T >= 2048) return go(std::integral_constant<int, 4>(), std::true_type(), std::false_type());
  return go(std::integral_constant<int, 2>(), std::true_type(), std::false_type());
}
