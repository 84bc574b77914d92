// moe_finalize_backward: gradients of the finalize (weighted sum of the top-k rows, shared
// row and residual, then the optional RMSNorm).
//
//   G = r (gamma dn - o r^2 mean(gamma dn o)) + dres,   r = 1 / sqrt(mean(o^2) + eps)
//   dy_j = w_j G,  dw_j = <G, y_j>,  dsum = G,  drms = sum_t dn o r
//
// Bound by HBM: a token moves 2 H (4 + 2 top_k) bytes and computes a few operations per
// element.  A CTA takes whole tokens (one CTA per SM for long rows); a producer thread streams the token's rows (dn, o,
// dres, then the top_k expert rows) by bulk copies into a ring of row slots, so that the next
// rows are on their way through the two block-wide sums of a token, and G stays in registers
// between them.  (Rows loaded by the threads themselves, two CTAs a SM: 28 KB in flight a SM and
// 3.0 TB/s; the ring has about 170 KB.)  drms: every thread owns the same columns for all tokens
// of its CTA and adds them in shared memory; one row of partial sums per CTA goes to the
// workspace and a second launch adds the rows in order (a fixed order: the same bits each time).
#include "moe_vec.cuh"

namespace moe {
namespace {

constexpr int kMaxConsumers = 512;
constexpr int kMaxK = 32;
constexpr int kMaxSlots = 16;
constexpr int kSmemMost = 225 * 1024;

struct FinBwd {
  const __nv_bfloat16 *dout, *dres, *o, *gamma, *y;
  const float* w;
  float eps;
  int T, H, k, slots;
  __nv_bfloat16 *dy, *dsum;
  float *dw, *partial;
};

__device__ __forceinline__ void bulk_load(void* smem_dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(smem_dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// blockDim.x = consumers + 32; consumers hold NV 8-element vectors of a row each.
template <int NV>
__global__ void __launch_bounds__(kMaxConsumers + 32, 1)
    finalize_backward_kernel(const FinBwd a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kMaxSlots], empty[kMaxSlots];
  __shared__ float red[2][kMaxConsumers / 32];
  __shared__ float dots[2][kMaxK][kMaxConsumers / 32];
  const int nvec = a.H / 8, consumers = blockDim.x - 32, warps = consumers >> 5;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t row_bytes = a.H * 2;
  float* drms_sum = reinterpret_cast<float*>(smem + (size_t)a.slots * row_bytes);  // [H] when partial
  depend_launch();
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.slots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], warps);
    }
    fence_mbar_init();
  }
  if (a.partial)
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) drms_sum[i] = 0.f;
  __syncthreads();

  if (warp == warps) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      // A consumer whose wait gave up hands slots back whose copies may still be on their way: none is filled,
      // and its barrier armed, again before the copy has landed (else it has long landed by then).
      auto push = [&](const __nv_bfloat16* row) {
        if (!ok || !(ok = mbar_wait(&empty[slot], phase ^ 1) && mbar_wait(&full[slot], phase ^ 1, false))) return;
        mbar_arrive_expect_tx(&full[slot], row_bytes);
        bulk_load(smem + (size_t)slot * row_bytes, row, row_bytes, &full[slot]);
        if (++slot == a.slots) {
          slot = 0;
          phase ^= 1;
        }
      };
      for (int t = blockIdx.x; t < a.T && ok; t += gridDim.x) {
        push(a.dout + (size_t)t * a.H);
        if (a.gamma) push(a.o + (size_t)t * a.H);
        if (a.dres) push(a.dres + (size_t)t * a.H);
        if (a.dw)
          for (int j = 0; j < a.k; ++j) push(a.y + ((size_t)t * a.k + j) * a.H);
      }
      // wait (bounded) for the copies still in flight before the shared memory goes: consumers that gave up
      // have not
      for (int i = 0; i < a.slots; ++i)
        mbar_wait(&full[i], i < slot ? phase : phase ^ 1, false, ok ? kWaitLimitNs : 100000000ull);
    }
  } else {
    // ------------------------------------------------------------ consumers
    // A wait that gives up (after two seconds, recorded) leaves wrong values but every barrier is
    // still met, so that all threads come to the end.
    int slot = 0;
    uint32_t phase = 0;
    auto take = [&]() {  // the next row, once it is there
      mbar_wait(&full[slot], phase);
      __syncwarp();
      return reinterpret_cast<const __nv_bfloat16*>(smem + (size_t)slot * row_bytes);
    };
    auto step = [&]() {
      if (++slot == a.slots) {
        slot = 0;
        phase ^= 1;
      }
    };
    auto done = [&](int s) {  // this warp has read slot s
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    };
    int par = 0;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x, par ^= 1) {
      float g[NV][8];
      const int s_dn = slot;
      const __nv_bfloat16* dn = take();
      step();
      if (a.gamma) {
        const int s_o = slot;
        const __nv_bfloat16* o = take();
        step();
        float sq = 0.f, gd = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int v = threadIdx.x + i * consumers;
          if (v >= nvec) continue;
          float d[8], x[8], gm[8];
          load8(dn + v * 8, d);
          load8(o + v * 8, x);
          load_bf16x8(a.gamma + v * 8, gm);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            sq += x[e] * x[e];
            gd += d[e] * gm[e] * x[e];
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
        named_bar_sync(1, consumers);
        sq = gd = 0.f;
        for (int i = 0; i < warps; ++i) {
          sq += red[0][i];
          gd += red[1][i];
        }
        const float r = __frsqrt_rn(sq / a.H + a.eps);
        const float c = r * r * (gd / a.H);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int v = threadIdx.x + i * consumers;
          if (v >= nvec) continue;
          float d[8], x[8], gm[8];
          load8(dn + v * 8, d);
          load8(o + v * 8, x);
          load_bf16x8(a.gamma + v * 8, gm);
          if (a.partial) {
            float4* m = reinterpret_cast<float4*>(drms_sum + v * 8);
            float4 lo = m[0], hi = m[1];
            lo.x += d[0] * x[0] * r, lo.y += d[1] * x[1] * r, lo.z += d[2] * x[2] * r, lo.w += d[3] * x[3] * r;
            hi.x += d[4] * x[4] * r, hi.y += d[5] * x[5] * r, hi.z += d[6] * x[6] * r, hi.w += d[7] * x[7] * r;
            m[0] = lo;
            m[1] = hi;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) g[i][e] = r * (d[e] * gm[e] - x[e] * c);
        }
        done(s_o);
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int v = threadIdx.x + i * consumers;
          if (v < nvec) load8(dn + v * 8, g[i]);
        }
      }
      done(s_dn);
      if (a.dres) {
        const int s_d = slot;
        const __nv_bfloat16* dr = take();
        step();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int v = threadIdx.x + i * consumers;
          if (v >= nvec) continue;
          float d[8];
          load8(dr + v * 8, d);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[i][e] += d[e];
        }
        done(s_d);
      }
      if (a.dsum) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int v = threadIdx.x + i * consumers;
          if (v < nvec) store8(a.dsum + (size_t)t * a.H + v * 8, g[i]);
        }
      }
      for (int j = 0; j < a.k; ++j) {
        const size_t row = ((size_t)t * a.k + j) * a.H;
        if (a.dy) {
          const float w = a.w ? __ldg(a.w + (size_t)t * a.k + j) : 1.f;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int v = threadIdx.x + i * consumers;
            if (v >= nvec) continue;
            float d[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = w * g[i][e];
            store8(a.dy + row + v * 8, d);
          }
        }
        if (a.dw) {
          const __nv_bfloat16* y = take();
          float dot = 0.f;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int v = threadIdx.x + i * consumers;
            if (v >= nvec) continue;
            float x[8];
            load8(y + v * 8, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) dot += g[i][e] * x[e];
          }
          done(slot);
          step();
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
          if (lane == 0) dots[par][j][warp] = dot;
        }
      }
      if (a.dw || a.gamma) named_bar_sync(1, consumers);  // (red is free again, dots are complete)
      if (a.dw && threadIdx.x < a.k) {
        float s = 0.f;
        for (int i = 0; i < warps; ++i) s += dots[par][threadIdx.x][i];
        a.dw[(size_t)t * a.k + threadIdx.x] = s;
      }
    }
    if (a.partial) {
      named_bar_sync(1, consumers);
      for (int i = threadIdx.x; i < a.H; i += consumers) a.partial[(size_t)blockIdx.x * a.H + i] = drms_sum[i];
    }
  }
}

// out[h] = sum over p of partial[p][h], p in ascending order within each of 8 interleaved sums.
__global__ void __launch_bounds__(256) drms_kernel(const float* __restrict__ partial, int P, int H, float* out) {
  __shared__ float sums[8][32];
  const int h = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  depend_wait();
  float s = 0.f;
  if (h < H)
#pragma unroll 8
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
// kMaxConsumers threads.
void shape(int H, int* consumers, int* nv) {
  const int nvec = H / 8;
  *nv = 1;
  while (nvec > *nv * kMaxConsumers) *nv *= 2;
  *consumers = ((nvec + *nv - 1) / *nv + 31) / 32 * 32;
}

// CTAs of an SM: short rows leave most of it idle between a token's sums, so several CTAs share it
// (within its registers: 95 a thread at most).  [2094, 416] top 4: one CTA an SM 40 us, eight under 10.
int ctas_per_sm(int H) {
  int consumers, nv;
  shape(H, &consumers, &nv);
  const int n = 65536 / (96 * (consumers + 32));
  return n < 1 ? 1 : n > 8 ? 8 : n;
}
int grid_ctas(int T, int H) {
  const int most = num_sms() * ctas_per_sm(H);
  return T < most ? T : most;
}

}  // namespace

MOE_DEFINE_STATUS_READER(finalize_backward_status)

}  // namespace moe

using namespace moe;

extern "C" size_t moe_finalize_backward_workspace_size(int T, int H) {
  if (T <= 0 || H <= 0) return 0;
  return (size_t)grid_ctas(T, H) * (size_t)H * sizeof(float);
}

extern "C" moe_status_t moe_finalize_backward(const void* dout, const void* dresidual_out, const void* residual_out,
                                              const void* rms_weight, float eps, const void* fused_expert_output,
                                              const float* topk_weights, int T, int H, int top_k, void* dy,
                                              float* dweights, void* dsum, float* drms, void* ws, size_t ws_bytes,
                                              moe_stream_t stream) {
  MOE_CHECK_ARG(T >= 0 && T <= (1 << 30) && H > 0 && H % 8 == 0 && top_k >= 1 && top_k <= kMaxK && eps >= 0.f);
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
  int consumers, nv;
  shape(H, &consumers, &nv);
  const int grid = grid_ctas(T, H);
  const size_t sums = drms ? (size_t)H * sizeof(float) : 0;
  a.slots = (int)(((size_t)kSmemMost / ctas_per_sm(H) - 5120 - sums) / ((size_t)H * 2));  // (5 KB: static)
  if (a.slots > kMaxSlots) a.slots = kMaxSlots;
  const size_t smem = sums + (size_t)a.slots * H * 2;
  auto run = [&](auto kern) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost - 5120) != cudaSuccess) return false;
    kern<<<grid, consumers + 32, smem, s>>>(a);
    return true;
  };
  const bool ok = nv == 1 ? run(finalize_backward_kernel<1>)
                          : nv == 2 ? run(finalize_backward_kernel<2>) : run(finalize_backward_kernel<4>);
  if (!ok) return MOE_ERR_CUDA;
  if (drms && launch_overlapped(drms_kernel, (H + 31) / 32, 256, s, a.partial, grid, H, drms) != cudaSuccess)
    return MOE_ERR_CUDA;
  return launch_status();
}
