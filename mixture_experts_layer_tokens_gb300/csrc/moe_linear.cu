// moe_linear and moe_linear_backward: D = A . B^T on the 5th-generation tensor cores with the
// projection's epilogue, and a dot-product kernel for a few rows.
//
//   forward   out [M, N] = act(x . w^T + bias) + residual     A = x  [M, K],  B = w [N, K]
//   dx [M, K] = dz . w                                        A = dz [M, N],  B = w^T
//   dw [N, K] = dz^T . x                                      A = dz^T,       B = x^T
//
// One kernel computes all three: an operand whose contraction dimension is contiguous is read
// "K-major", the transposed ones "MN-major" straight from the same row-major tensors (the
// tensor core takes either order from shared memory), so nothing is transposed in memory.
//
// Persistent, warp-specialised: warp 0 copies 64-deep K blocks of A and B by TMA into a ring
// of stages, warp 1 issues the MMAs from one lane into one of two accumulators in tensor
// memory, warps 2-5 (one per 32 TMEM lanes) take the other accumulator through the epilogue.
// Problems with fewer tiles than SMs split K over the CTAs of a thread-block cluster: each
// leaves its fp32 partial tile in its own shared memory, and after one cluster barrier every
// CTA adds its share of the elements over distributed shared memory, in rank order.
#include "moe_vec.cuh"

#include <cudaTypedefs.h>

namespace moe {
namespace {

constexpr int BM = 128;           // accumulator rows of a CTA = TMEM lanes
constexpr int BK = 64;            // contraction elements of a stage: one 128-byte swizzle row
constexpr int kThreads = 192;     // producer, MMA issuer, 4 epilogue warps
constexpr int kEpiWarps = 4;
constexpr int kMaxStages = 8;
constexpr int kStageBudget = 192 * 1024;
constexpr int kBufStride = 36;    // floats: 32 columns of a row, padded so that 16-byte accesses hit distinct banks
constexpr int kBufBytes = kEpiWarps * 32 * kBufStride * 4;
constexpr int kSmemBytes = 1024 + kStageBudget + kBufBytes + 1024;
constexpr int kTmemCols = 512;
constexpr int kAccCols = 256;     // columns between the two accumulators

__device__ __forceinline__ float act_fwd(float z, int act) {
  switch (act) {
    case MOE_LINEAR_SILU: return __fdividef(z, 1.0f + expf(-z));
    case MOE_LINEAR_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678f));
    case MOE_LINEAR_GELU_TANH: return 0.5f * z * (1.0f + tanhf(0.79788456f * (z + 0.044715f * z * z * z)));
  }
  return z;
}

__device__ __forceinline__ float act_grad(float z, int act) {
  switch (act) {
    case MOE_LINEAR_SILU: {
      const float q = __fdiv_rn(1.0f, 1.0f + expf(-z));
      return q * (1.0f + z * (1.0f - q));
    }
    case MOE_LINEAR_GELU:
      return 0.5f * (1.0f + erff(z * 0.70710678f)) + z * 0.39894228f * expf(-0.5f * z * z);
    case MOE_LINEAR_GELU_TANH: {
      const float t = tanhf(0.79788456f * (z + 0.044715f * z * z * z));
      return 0.5f * (1.0f + t) + 0.5f * z * (1.0f - t * t) * 0.79788456f * (1.0f + 0.134145f * z * z);
    }
  }
  return 1.0f;
}

// What is done with a sum z at (row, col) of D [P, Q].
struct Epilogue {
  const void* bias;
  const void* residual;
  void* out;
  void* preact;
  int P, Q;
  int act;
  int fp16;   // 16-bit values are fp16 (else bf16)
  int out32;  // out and residual are fp32
};

__device__ __forceinline__ float load16(const void* p, size_t i, int fp16) {
  return fp16 ? load1(static_cast<const __half*>(p) + i) : load1(static_cast<const __nv_bfloat16*>(p) + i);
}
__device__ __forceinline__ void store16(void* p, size_t i, float v, int fp16) {
  if (fp16)
    store1(static_cast<__half*>(p) + i, v);
  else
    store1(static_cast<__nv_bfloat16*>(p) + i, v);
}

__device__ __forceinline__ void finish1(const Epilogue& e, int row, int col, float z) {
  const size_t at = (size_t)row * e.Q + col;
  if (e.bias) z += load16(e.bias, col, e.fp16);
  if (e.preact) store16(e.preact, at, z, e.fp16);
  z = act_fwd(z, e.act);
  // (residual may be out: a plain load, not the read-only path)
  if (e.out32) {
    if (e.residual) z += static_cast<const float*>(e.residual)[at];
    static_cast<float*>(e.out)[at] = z;
  } else {
    if (e.residual)
      z += e.fp16 ? __half2float(static_cast<const __half*>(e.residual)[at])
                  : __bfloat162float(static_cast<const __nv_bfloat16*>(e.residual)[at]);
    store16(e.out, at, z, e.fp16);
  }
}

template <class T>
__device__ __forceinline__ void add8(const void* p, size_t at, float (&z)[8]) {
  float v[8];
  load8(static_cast<const T*>(p) + at, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] += v[i];
}

// 8 consecutive columns of a row (Q % 8 == 0).
__device__ __forceinline__ void finish8(const Epilogue& e, int row, int col, float (&z)[8]) {
  const size_t at = (size_t)row * e.Q + col;
  if (e.bias) {
    if (e.fp16)
      add8<__half>(e.bias, col, z);
    else
      add8<__nv_bfloat16>(e.bias, col, z);
  }
  if (e.preact) {
    if (e.fp16)
      store8(static_cast<__half*>(e.preact) + at, z);
    else
      store8(static_cast<__nv_bfloat16*>(e.preact) + at, z);
  }
  if (e.act != MOE_LINEAR_NONE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_fwd(z[i], e.act);
  }
  if (e.out32) {
    if (e.residual) add8<float>(e.residual, at, z);
    store8(static_cast<float*>(e.out) + at, z);
  } else if (e.fp16) {
    if (e.residual) add8<__half>(e.residual, at, z);
    store8(static_cast<__half*>(e.out) + at, z);
  } else {
    if (e.residual) add8<__nv_bfloat16>(e.residual, at, z);
    store8(static_cast<__nv_bfloat16*>(e.out) + at, z);
  }
}

// ------------------------------------------------------------------ tensor-core kernel
struct Gemm {
  Epilogue e;
  int KB;               // K blocks
  int splits;           // CTAs (of a cluster) that share a tile's K blocks
  int BN;               // tile columns
  int stages;
  int a_rows;           // rows of the A box (K-major A)
  int tiles_m, tiles_n;
  uint32_t idesc;
};

// Shared-memory descriptor of an MN-major operand as TMA boxes of 64 MN elements x 64 K
// elements write it with 128-byte swizzle: rows of 128 bytes along MN, 8 K rows per 1024-byte
// atom (stride offset), consecutive 64-element MN groups 8 KB apart (leading offset).
__device__ __forceinline__ uint64_t mn_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFF) >> 4);
  d |= (uint64_t)(8192 >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t smem_addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr), "r"(rank));
  return a;
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// The tile of a unit: blocks of kRaster tile rows run through all tile columns, so that the
// CTAs that work at the same time share A rows and B rows in L2.
constexpr int kRaster = 8;
__device__ __forceinline__ void tile_of(int u, int tiles_m, int tiles_n, int& m, int& n) {
  const int per = kRaster * tiles_n, g = u / per, in = u - g * per;
  const int rows = min(kRaster, tiles_m - g * kRaster);
  m = g * kRaster + in % rows;
  n = in / rows;
}

// kAMN / kBMN: the operand is MN-major (its contraction dimension is the row of its tensor).
template <bool kAMN, bool kBMN>
__global__ void __launch_bounds__(kThreads, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ Gemm p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ctrl = smem + kStageBudget;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;  // [2] accumulator complete
  uint64_t* tempty = tfull + 2;          // [2] accumulator read
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  float* bufs = reinterpret_cast<float*>(ctrl + 1024);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = p.stages;
  const uint32_t a_bytes = kAMN ? 128 * BK * 2 : p.a_rows * 128;
  const uint32_t b_bytes = p.BN * 128;
  const int stage_bytes = 128 * 128 + p.BN * 128;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kEpiWarps);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    prefetch_tensormap(&tmA);
    prefetch_tensormap(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int splits = p.splits;
  const int rank = splits > 1 ? (int)cluster_rank() : 0;
  const int kb0 = (int)((long long)p.KB * rank / splits), kb1 = (int)((long long)p.KB * (rank + 1) / splits);
  const int units = p.tiles_m * p.tiles_n;
  const int first = splits > 1 ? blockIdx.x / splits : blockIdx.x;
  const int step = splits > 1 ? units : gridDim.x;  // a split tile is its cluster's only work

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    const uint64_t pol = policy_evict_normal();
    int stage = 0;
    uint32_t phase = 0;
    long long fills = 0;
    bool ok = true;
    for (int u = first; ok && u < units; u += step) {
      int tm, tn;
      tile_of(u, p.tiles_m, p.tiles_n, tm, tn);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(ok = warp_wait(&empty[stage], phase ^ 1))) break;
        if (lane == 0) {
          uint8_t* sA = smem + stage * stage_bytes;
          uint8_t* sB = sA + 128 * 128;
          mbar_arrive_expect_tx(&full[stage], a_bytes + b_bytes);
          if (kAMN) {
            tma_load_2d(sA, &tmA, tm * BM, kb * BK, &full[stage], pol);
            tma_load_2d(sA + 8192, &tmA, tm * BM + 64, kb * BK, &full[stage], pol);
          } else {
            tma_load_2d(sA, &tmA, kb * BK, tm * BM, &full[stage], pol);
          }
          if (kBMN) {
            for (int g = 0; g < p.BN / 64; ++g)
              tma_load_2d(sB + g * 8192, &tmB, tn * p.BN + g * 64, kb * BK, &full[stage], pol);
          } else {
            tma_load_2d(sB, &tmB, kb * BK, tn * p.BN, &full[stage], pol);
          }
        }
        __syncwarp();
        ++fills;
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (status_failed() && lane == 0) {
      // wait (bounded) for the copies still in flight: the last fill of each stage
      for (long long i = fills - 1; i >= 0 && i >= fills - stages; --i)
        mbar_wait(&full[i % stages], (uint32_t)((i / stages) & 1), false, 100000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int u = first; ok && u < units; u += step) {
      if (!(ok = warp_wait(&tempty[acc], acc_phase ^ 1))) break;
      tc_fence_after();
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(ok = warp_wait(&full[stage], phase))) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t a0 = smem_u32(smem + stage * stage_bytes), b0 = a0 + 128 * 128;
          const uint32_t d = tmem + acc * kAccCols;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t ad = kAMN ? mn_desc(a0 + kk * 2048) : sw128_desc(a0 + kk * 32);
            const uint64_t bd = kBMN ? mn_desc(b0 + kk * 2048) : sw128_desc(b0 + kk * 32);
            mma_bf16(d, ad, bd, p.idesc, kb > kb0 || kk > 0);
          }
          tc_commit(&empty[stage]);
        }
        __syncwarp();
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (ok) {
        if (lane == 0) tc_commit(&tfull[acc]);
        __syncwarp();
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
    }
    if (!ok) {
      // a wait gave up: let the MMAs issued so far finish (bounded) before the tensor memory goes
      if (lane == 0) {
        tc_commit(drain);
        mbar_wait(drain, 0, false, 100000000ull);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;  // TMEM lanes this warp may access
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    float* buf = bufs + (warp - 2) * 32 * kBufStride;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int u = first; u < units; u += step) {
      int tm, tn;
      tile_of(u, p.tiles_m, p.tiles_n, tm, tn);
      if (!warp_wait(&tfull[acc], acc_phase)) break;
      tc_fence_after();
      const uint32_t tb = tmem + lane_addr + acc * kAccCols;
      const int row0 = tm * BM + quarter * 32, col0 = tn * p.BN;
      const int cols = min(p.BN, p.e.Q - col0);
      if (splits > 1) {
        // the whole partial tile into this CTA's stages: every copy has landed and every MMA
        // has read it
        float* part = reinterpret_cast<float*>(smem) + (quarter * 32 + lane) * (p.BN + 4);
        if (row0 < p.e.P)
          for (int c = 0; c < cols; c += 32) {
            float v[32];
            tmem_ld32(tb + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(part + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
      } else {
        if (row0 < p.e.P)
          for (int c = 0; c < cols; c += 32) {
            float v[32];
            tmem_ld32(tb + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(buf + lane * kBufStride + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            __syncwarp();
            if (p.e.Q % 8 == 0) {
              // 4 lanes to the 32 columns of a row: 64-byte pieces of 8 rows at a time
              const int col = col0 + c + (lane & 3) * 8;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = i * 8 + (lane >> 2);
                if (row0 + r < p.e.P && col < p.e.Q) {
                  const float4 lo = *reinterpret_cast<const float4*>(buf + r * kBufStride + (lane & 3) * 8);
                  const float4 hi = *reinterpret_cast<const float4*>(buf + r * kBufStride + (lane & 3) * 8 + 4);
                  float z[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                  finish8(p.e, row0 + r, col, z);
                }
              }
            } else {
              for (int r = 0; r < 32 && row0 + r < p.e.P; ++r)
                if (col0 + c + lane < p.e.Q) finish1(p.e, row0 + r, col0 + c + lane, buf[r * kBufStride + lane]);
            }
            __syncwarp();
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc]);
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
  }

  if (splits > 1) {
    __syncwarp();
    cluster_sync();  // every CTA's partial tile is in its shared memory
    int tm, tn;
    tile_of(first, p.tiles_m, p.tiles_n, tm, tn);
    const int rows = min(BM, p.e.P - tm * BM), cols = min(p.BN, p.e.Q - tn * p.BN);
    const int groups = (cols + 7) / 8, items = rows * groups;
    const uint32_t base = smem_u32(smem);
    const int i1 = (int)((long long)items * (rank + 1) / splits);
    if (!status_failed())
      for (int i = (int)((long long)items * rank / splits) + threadIdx.x; i < i1; i += kThreads) {
        const int r = i / groups, c = (i - r * groups) * 8;
        const uint32_t at = base + (uint32_t)((r * (p.BN + 4) + c) * 4);
        float z[8] = {};
        for (int s = 0; s < splits; ++s) {
          const uint32_t src = map_to_rank(at, s);
          const float4 lo = ld_cluster(src), hi = ld_cluster(src + 16);
          z[0] += lo.x, z[1] += lo.y, z[2] += lo.z, z[3] += lo.w;
          z[4] += hi.x, z[5] += hi.y, z[6] += hi.z, z[7] += hi.w;
        }
        const int row = tm * BM + r, col = tn * p.BN + c;
        if (p.e.Q % 8 == 0) {
          finish8(p.e, row, col, z);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (col + j < p.e.Q) finish1(p.e, row, col + j, z[j]);
        }
      }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another reads its shared memory
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ a few rows
// out [M, N] for M <= kM: each warp takes one weight row (or 1/KS of it) and all M rows of x.
// Bound by the weights' bytes; a lane's loads are independent, so a CTA has the whole of its
// weight slice in flight.
template <int kM, class T>
__global__ void __launch_bounds__(256)
    linear_rows_kernel(const T* __restrict__ x, const T* __restrict__ w, int M, int N, int K, int ks, const Epilogue e) {
  __shared__ float sums[8][kM];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = 8 / ks;  // weight rows of the CTA
  const int n = blockIdx.x * per + warp / ks, part = warp % ks;
  float acc[kM] = {};
  if (n < N) {
    const T* wr = w + (size_t)n * K;
#pragma unroll 4
    for (int k = (part * 32 + lane) * 8; k < K; k += ks * 256) {
      float wv[8];
      load8(wr + k, wv);
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        if (m >= M) break;
        float xv[8];
        load8(x + (size_t)m * K + k, xv);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[m] = fmaf(wv[i], xv[i], acc[m]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < kM; ++m) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) acc[m] += __shfl_xor_sync(0xffffffffu, acc[m], off);
    if (lane == 0) sums[warp][m] = acc[m];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < per * M; i += blockDim.x) {
    const int r = i % per, m = i / per, col = blockIdx.x * per + r;
    if (col >= N) continue;
    float z = 0.f;
    for (int s = 0; s < ks; ++s) z += sums[r * ks + s][m];
    finish1(e, m, col, z);
  }
}

// ------------------------------------------------------------------ dz and its column sums
// dz = dout * act'(preact), in the operand type (row stride ld), and one row of column sums per
// chunk of rows.  A thread takes 8 columns (or 1 where N % 8) of every 8th row of its chunk.
constexpr int kDzRows = 64;       // rows of a chunk, more where that would give over
constexpr int kDzChunks = 1024;   // this many

template <class TO, class T, bool kVec>
__global__ void __launch_bounds__(256)
    linear_dz_kernel(const TO* __restrict__ dout, const T* __restrict__ preact, int M, int N, int act, T* __restrict__ dz,
                     int ld, int rows, float* __restrict__ partial) {
  constexpr int V = kVec ? 8 : 1;
  __shared__ float sums[8][32 * V];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int col = (blockIdx.x * 32 + cx) * V;
  const int r0 = blockIdx.y * rows, r1 = min(M, r0 + rows);
  float sum[V] = {};
  if (col < N)
    for (int r = r0 + ry; r < r1; r += 8) {
      const size_t at = (size_t)r * N + col;
      float d[V];
      if constexpr (kVec)
        load8(dout + at, d);
      else
        d[0] = load1(dout + at);
      if (act != MOE_LINEAR_NONE) {
        float z[V];
        if constexpr (kVec)
          load8(preact + at, z);
        else
          z[0] = load1(preact + at);
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] *= act_grad(z[i], act);
      }
      if (dz) {
        if constexpr (kVec)
          store8(dz + (size_t)r * ld + col, d);
        else
          store1(dz + (size_t)r * ld + col, d[0]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += d[i];
    }
  if (!partial) return;
#pragma unroll
  for (int i = 0; i < V; ++i) sums[ry][cx * V + i] = sum[i];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * V; i += 256) {
    const int c = blockIdx.x * 32 * V + i;
    float s = 0.f;
    for (int y = 0; y < 8; ++y) s += sums[y][i];
    if (c < N) partial[(size_t)blockIdx.y * N + c] = s;
  }
}

template <class T>
__global__ void __launch_bounds__(256) linear_dbias_kernel(const float* __restrict__ partial, int P, int N, T* dbias) {
  __shared__ float sums[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  float s = 0.f;
  if (c < N)
    for (int p = part; p < P; p += 8) s += partial[(size_t)p * N + c];
  sums[part][threadIdx.x & 31] = s;
  __syncthreads();
  if (part == 0 && c < N) {
    for (int i = 1; i < 8; ++i) s += sums[i][threadIdx.x & 31];
    store1(dbias + c, s);
  }
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}

// A 16-bit row-major tensor [rows][inner] with row stride ld (elements), read in boxes of 64
// inner elements x box_rows rows.
bool make_map(CUtensorMap* m, const void* base, int fp16, long long inner, long long rows, long long ld, int box_rows) {
  auto enc = get_encode();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(ld * 2)};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Operand {
  const void* base;
  bool mn;  // MN-major: the tensor's rows are the contraction
  long long ld;
};

int cdiv(long long a, long long b) { return (int)((a + b - 1) / b); }

template <bool kAMN, bool kBMN>
cudaError_t launch_gemm(const CUtensorMap& ma, const CUtensorMap& mb, const Gemm& g, int grid, cudaStream_t s) {
  auto kern = linear_gemm_kernel<kAMN, kBMN>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = g.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, ma, mb, g);
}

// D [P, Q] = A . B^T over a contraction of C.
moe_status_t run_gemm(const Operand& A, const Operand& B, int C, const Epilogue& e, cudaStream_t s) {
  Gemm g;
  g.e = e;
  g.KB = cdiv(C, BK);
  const int nsm = num_sms();
  g.tiles_m = cdiv(e.P, BM);
  int bn = 256;
  while (bn > 64 && (bn / 2 >= e.Q || g.tiles_m * cdiv(e.Q, bn) * 2 <= nsm)) bn /= 2;
  g.BN = bn;
  g.tiles_n = cdiv(e.Q, bn);
  const long long units = (long long)g.tiles_m * g.tiles_n;
  if (units > 2147483647LL / 8) return MOE_ERR_UNSUPPORTED;
  int S = 1;
  while (S < 8 && units * S * 2 <= nsm && g.KB / (2 * S) >= 4) S *= 2;
  g.splits = S;
  g.stages = kStageBudget / (128 * 128 + bn * 128);
  if (g.stages > kMaxStages) g.stages = kMaxStages;
  g.a_rows = e.P >= BM ? BM : (e.P + 7) / 8 * 8;
  g.idesc = make_idesc(e.fp16 ? 0 : 1, BM, bn) | (A.mn ? 1u << 15 : 0) | (B.mn ? 1u << 16 : 0);
  CUtensorMap ma, mb;
  const bool ok = (A.mn ? make_map(&ma, A.base, e.fp16, e.P, C, A.ld, BK)
                        : make_map(&ma, A.base, e.fp16, C, e.P, A.ld, g.a_rows)) &&
                  (B.mn ? make_map(&mb, B.base, e.fp16, e.Q, C, B.ld, BK)
                        : make_map(&mb, B.base, e.fp16, C, e.Q, B.ld, bn));
  if (!ok) return MOE_ERR_CUDA;
  const int grid = S > 1 ? (int)units * S : (int)(units < nsm ? units : nsm);
  const cudaError_t err = A.mn ? launch_gemm<true, true>(ma, mb, g, grid, s)
                          : B.mn ? launch_gemm<false, true>(ma, mb, g, grid, s)
                                 : launch_gemm<false, false>(ma, mb, g, grid, s);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int kM>
void launch_rows(const void* x, const void* w, int M, int N, int K, const Epilogue& e, cudaStream_t s) {
  int ks = 1;
  while (ks < 8 && (long long)N * ks < 16LL * num_sms() && ks * 512 <= K) ks *= 2;
  const int grid = cdiv(N, 8 / ks);
  if (e.fp16)
    linear_rows_kernel<kM, __half>
        <<<grid, 256, 0, s>>>(static_cast<const __half*>(x), static_cast<const __half*>(w), M, N, K, ks, e);
  else
    linear_rows_kernel<kM, __nv_bfloat16>
        <<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(w), M, N, K, ks, e);
}

struct BwdLayout {
  long long ld;
  int rows, chunks;  // of linear_dz_kernel
  size_t partial, total;
};
BwdLayout bwd_layout(int M, int N) {
  BwdLayout l;
  l.ld = ((long long)N + 7) / 8 * 8;
  l.rows = kDzRows;
  while (cdiv(M, l.rows) > kDzChunks) l.rows *= 2;
  l.chunks = cdiv(M, l.rows);
  l.partial = ((size_t)M * l.ld * 2 + 255) / 256 * 256;
  l.total = l.partial + (size_t)l.chunks * N * sizeof(float);
  return l;
}

template <class TO, class T>
void launch_dz(const void* dout, const void* preact, int M, int N, int act, void* dz, const BwdLayout& l, float* partial,
               cudaStream_t s) {
  const TO* d = static_cast<const TO*>(dout);
  const T* z = static_cast<const T*>(preact);
  if (N % 8 == 0)
    linear_dz_kernel<TO, T, true><<<dim3(cdiv(N, 256), l.chunks), 256, 0, s>>>(d, z, M, N, act, static_cast<T*>(dz),
                                                                               (int)l.ld, l.rows, partial);
  else
    linear_dz_kernel<TO, T, false><<<dim3(cdiv(N, 32), l.chunks), 256, 0, s>>>(d, z, M, N, act, static_cast<T*>(dz),
                                                                               (int)l.ld, l.rows, partial);
}

moe_status_t check_sizes(int M, int N, int K, moe_dtype_t dtype, int activation, moe_dtype_t other) {
  MOE_CHECK_ARG(M >= 0 && N >= 1 && K >= 8 && K % 8 == 0);
  MOE_CHECK_ARG(M <= (1 << 30) && N <= (1 << 21) && K <= (1 << 30));
  if (dtype != MOE_DT_BF16 && dtype != MOE_DT_FP16) return MOE_ERR_UNSUPPORTED;
  if (other != dtype && other != MOE_DT_FP32) return MOE_ERR_UNSUPPORTED;
  if (activation < MOE_LINEAR_NONE || activation > MOE_LINEAR_GELU_TANH) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

MOE_DEFINE_STATUS_READER(linear_status)

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_linear(const void* x, const void* w, const void* bias, const void* residual, int M, int N,
                                   int K, moe_dtype_t dtype, int activation, moe_dtype_t out_dtype, void* out,
                                   void* preact, moe_stream_t stream) {
  const moe_status_t st = check_sizes(M, N, K, dtype, activation, out_dtype);
  if (st != MOE_OK) return st;
  if (M == 0) return MOE_OK;
  MOE_CHECK_ARG(x && w && out);
  MOE_CHECK_ARG(aligned16(x) && aligned16(w) && aligned16(bias) && aligned16(residual) && aligned16(out) &&
                aligned16(preact));
  const Epilogue e{bias, residual, out, preact, M, N, activation, dtype == MOE_DT_FP16, out_dtype == MOE_DT_FP32};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M <= 4) {
    if (M == 1)
      launch_rows<1>(x, w, M, N, K, e, s);
    else if (M == 2)
      launch_rows<2>(x, w, M, N, K, e, s);
    else
      launch_rows<4>(x, w, M, N, K, e, s);
    return launch_status();
  }
  return run_gemm({x, false, K}, {w, false, K}, K, e, s);
}

extern "C" size_t moe_linear_backward_workspace_size(int M, int N, int K) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  return bwd_layout(M, N).total;
}

extern "C" moe_status_t moe_linear_backward(const void* dout, moe_dtype_t dout_dtype, const void* x, const void* w,
                                            const void* preact, int M, int N, int K, moe_dtype_t dtype, int activation,
                                            void* dx, void* dw, void* dbias, void* ws, size_t ws_bytes,
                                            moe_stream_t stream) {
  moe_status_t st = check_sizes(M, N, K, dtype, activation, dout_dtype);
  if (st != MOE_OK) return st;
  MOE_CHECK_ARG(dx || dw || dbias);
  MOE_CHECK_ARG(aligned16(dx) && aligned16(dw) && aligned16(dbias));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {
    if (dw && cudaMemsetAsync(dw, 0, (size_t)N * K * 2, s) != cudaSuccess) return MOE_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, (size_t)N * 2, s) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  MOE_CHECK_ARG(dout && (!dx || w) && (!dw || x) && (preact || activation == MOE_LINEAR_NONE));
  MOE_CHECK_ARG(aligned16(dout) && aligned16(x) && aligned16(w) && aligned16(preact) && aligned16(ws));
  if (!ws || ws_bytes < moe_linear_backward_workspace_size(M, N, K)) return MOE_ERR_WORKSPACE;
  const BwdLayout l = bwd_layout(M, N);
  const int fp16 = dtype == MOE_DT_FP16;
  // dout itself is the operand when it needs no arithmetic, no rounding and TMA can read its rows
  const bool direct = activation == MOE_LINEAR_NONE && dout_dtype == dtype && N % 8 == 0;
  void* dz = (direct || !(dx || dw)) ? nullptr : ws;
  float* partial = dbias ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + l.partial) : nullptr;
  if (dz || partial) {
    if (fp16) {
      if (dout_dtype == MOE_DT_FP32)
        launch_dz<float, __half>(dout, preact, M, N, activation, dz, l, partial, s);
      else
        launch_dz<__half, __half>(dout, preact, M, N, activation, dz, l, partial, s);
    } else {
      if (dout_dtype == MOE_DT_FP32)
        launch_dz<float, __nv_bfloat16>(dout, preact, M, N, activation, dz, l, partial, s);
      else
        launch_dz<__nv_bfloat16, __nv_bfloat16>(dout, preact, M, N, activation, dz, l, partial, s);
    }
    if (dbias) {
      if (fp16)
        linear_dbias_kernel<<<cdiv(N, 32), 256, 0, s>>>(partial, l.chunks, N, static_cast<__half*>(dbias));
      else
        linear_dbias_kernel<<<cdiv(N, 32), 256, 0, s>>>(partial, l.chunks, N, static_cast<__nv_bfloat16*>(dbias));
    }
    if ((st = launch_status()) != MOE_OK) return st;
  }
  const void* z = direct ? dout : dz;
  const long long ld = direct ? N : l.ld;
  if (dx) {
    const Epilogue e{nullptr, nullptr, dx, nullptr, M, K, MOE_LINEAR_NONE, fp16, 0};
    if ((st = run_gemm({z, false, ld}, {w, true, K}, N, e, s)) != MOE_OK) return st;
  }
  if (dw) {
    const Epilogue e{nullptr, nullptr, dw, nullptr, N, K, MOE_LINEAR_NONE, fp16, 0};
    if ((st = run_gemm({z, true, ld}, {x, true, K}, M, e, s)) != MOE_OK) return st;
  }
  return launch_status();
}
