// moe_grouped_linear and moe_grouped_linear_backward: the experts' products over ragged groups of rows, on the
// 5th-generation tensor cores.  The sorted rows p of expert e are [offsets[e], offsets[e + 1]):
//
//   forward  out_p = w_e x_p            [N] over K
//   dx       dx_p  = w_e^T dout_p       [K] over N
//   dw       dw_e  = sum_p dout_p x_p^T [N, K] over the group's rows
//
// Bound by the tensor cores (2 N K a row and product) where a group has some 300 rows or more, by the
// weights' bytes below.  Forward and dx put the weights on the MMA's 256 rows (a pair of CTAs, 128 each) and the
// group's rows on its columns: a tile has as many columns as its group has rows left, in steps of 32, so a
// ragged group wastes 16 columns on the average where tiles of 128 rows of it waste 64, and a decoded
// token's experts read their weights once over narrow tiles.  dw has no ragged side but its contraction: 64 rows
// at a time, and in the group's last block the rows behind its end (the next expert's) are zeroed in
// shared memory before the MMAs see them.
//
// Persistent, warp-specialised, pairs of CTAs: warp 0 copies stages of K blocks by TMA, warp 1 issues the MMAs, warps
// 2 and 3 zero dw's tails, warps 4-11 run the epilogue from one of two accumulators in tensor memory while the
// other fills.  Every CTA counts the tiles from the offsets itself; nothing comes back to the host.
#include "moe_mma.cuh"

#include <atomic>

namespace moe {
namespace {

constexpr int BK = 64;            // contraction elements of a K block: one 128-byte swizzle row
constexpr int kRows = 128;        // rows of A of a CTA
constexpr int kThreads = 384;
constexpr int kFirstEpi = 4;
constexpr int kEpiWarps = 8;
constexpr int kMaxStages = 8;
constexpr int kMaxE = 1024;
constexpr int kStageBudget = 192 * 1024;
constexpr int kCtrlBytes = 512;
constexpr int kBufBytes = 2048;   // of an epilogue warp
constexpr int kTableBytes = 2 * (kMaxE + 4) * 4;
constexpr int kSmemBytes = 1024 + kStageBudget + kCtrlBytes + kEpiWarps * kBufBytes + kTableBytes;
// K blocks of a sum in tensor memory, whose additions truncate, by the output's type; longer ones are added up in
// fp32 registers with rounding (kPromote), as moe_linear's are
constexpr int kRunFP32 = 8, kRunFP16 = 128, kRunBF16 = 256;
constexpr int kLaunchRegs = 168, kLowRegs = 40, kHighRegs = 232;
static_assert(128 * kLowRegs + 256 * kHighRegs == kThreads * kLaunchRegs, "register split must balance");
static_assert((4 * kMaxStages + 5) * 8 + 4 <= kCtrlBytes && kSmemBytes <= 232448, "shared memory layout");

enum Mode { kForward, kDx, kDw };

struct Grouped {
  const int32_t *offsets, *slots;  // slots: rows of out are the slots of the sorted rows (NULL: the sorted rows)
  void* out;
  int S, E;
  int P, Q;              // rows of A's tensor (forward N, dx K, dw N); dw: columns of B's (K)
  int KB;                // stages of the contraction (dw: by the group's rows)
  int tiles_p, tiles_q;  // of 256 rows of A; dw: of `width` columns
  int width;             // columns of a tile at most
  int box;               // rows of a box of B (forward and dx)
  int stages, chunk;     // chunk: stages added up in the tensor memory (kPromote)
  int fp16, out32, accumulate;
  uint32_t idesc;        // but for the columns
};

struct Unit {
  int p, q;        // tile of A; dw: of B
  int row0, rows;  // sorted rows: of the tile (forward, dx), of the group (dw)
  int width;       // columns of the tile
  int stages;      // of its contraction
  long long e;
};

// Tile of the unit u.  Blocks of up to 8 tile columns run through all tile rows (dw: the other way round), so that
// the pairs that work at the same time share both operands in L2.
constexpr int kRaster = 8;
__device__ __forceinline__ void raster(int in, int many, int other, int& a, int& b) {
  const int blocks = (many + kRaster - 1) / kRaster, r = (many + blocks - 1) / blocks;
  const int g = in / (r * other), left = in - g * r * other, n = min(r, many - g * r);
  a = g * r + left % n;
  b = left / n;
}
template <Mode kMode>
__device__ __forceinline__ Unit unit_of(const Grouped& p, const int* start, const int* pre, int u) {
  Unit t;
  if constexpr (kMode == kDw) {
    const int per = p.tiles_p * p.tiles_q, e = u / per;
    raster(u - e * per, p.tiles_p, p.tiles_q, t.p, t.q);
    t.e = e;
    t.row0 = start[e];
    t.rows = max(0, start[e + 1] - t.row0);
    t.width = p.width;
    t.stages = (t.rows + BK - 1) / BK;
  } else {
    const int at = u / p.tiles_p;
    int e = 0, end = p.E;  // the last e with pre[e] <= at
    while (end - e > 1) {
      const int mid = (e + end) >> 1;
      if (pre[mid] <= at)
        e = mid;
      else
        end = mid;
    }
    const int n = pre[e + 1] - pre[e], rows = start[e + 1] - start[e];
    raster(u - p.tiles_p * pre[e], n, p.tiles_p, t.q, t.p);
    t.e = e;
    // the group's rows dealt evenly over its tiles (that many are needed, so none is empty)
    t.width = ((rows + n - 1) / n + 31) & ~31;
    t.row0 = start[e] + t.q * t.width;
    t.rows = min(t.width, rows - t.q * t.width);
    t.stages = p.KB;
  }
  return t;
}

__device__ __forceinline__ void tma_load_pair_3d(void* smem_dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}
// lane_wait that also acquires what the other CTA of the pair released.
__device__ __forceinline__ bool lane_wait_cluster(uint64_t* bar, uint32_t parity) {
  if (!lane_wait(bar, parity)) return false;
  uint32_t ok;  // (the phase is over: one test)
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack16(float a, float b, int fp16) {
  const float v[2] = {a, b};
  return fp16 ? Word<__half>::put(v) : Word<__nv_bfloat16>::put(v);
}

// 32 rows of A (lanes, from n0) x 32 sorted rows (v, from row0, `rows` of them valid) into out, 16 bits, transposed
// through the warp's buffer: lanes pair up so that a word holds two neighbouring columns of out.
__device__ __forceinline__ void store_rows32(const Grouped& p, char* buf, const float* v, int n0, int row0, int rows,
                                             int lane) {
  uint32_t* words = reinterpret_cast<uint32_t*>(buf);
  const bool odd = lane & 1;
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    const uint32_t mine = pack16(v[c], v[c + 1], p.fp16), other = __shfl_xor_sync(0xffffffffu, mine, 1);
    words[(c + odd) * 16 + (lane >> 1)] = odd ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x5410);
  }
  __syncwarp();
  const int piece = lane & 3, col = n0 + piece * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = i * 8 + (lane >> 2);
    if (c < rows && col < p.P) {
      long long row = row0 + c;
      if (p.slots) {
        row = p.slots[row];
        if (row < 0 || row >= p.S) {
          record_status((int)MOE_ERR_INVALID_ARG);
          continue;
        }
      }
      const uint4 w = *reinterpret_cast<const uint4*>(buf + c * 64 + piece * 16);
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * p.P + col) = w;
    }
  }
  __syncwarp();
}

// 32 rows (lanes, from n0) x 32 columns (v, from k0) of an expert's weight gradient at `out`.
__device__ __forceinline__ void store_grad32(const Grouped& p, char* buf, const float* v, size_t out, int n0, int k0, int lane) {
  auto at = [&](int row, int piece) { return buf + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4); };
  const int piece = lane & 3;
  if (!p.out32 && !p.accumulate) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack16(v[8 * i + 2 * j], v[8 * i + 2 * j + 1], p.fp16);
      *reinterpret_cast<uint4*>(at(lane, i)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
    const int col = k0 + piece * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + (lane >> 2);
      if (n0 + r < p.P && col < p.Q)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + out + (size_t)(n0 + r) * p.Q + col) =
            *reinterpret_cast<const uint4*>(at(r, piece));
    }
    __syncwarp();
    return;
  }
#pragma unroll
  for (int h = 0; h < 32; h += 16) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(at(lane, i)) =
          make_float4(v[h + 4 * i], v[h + 4 * i + 1], v[h + 4 * i + 2], v[h + 4 * i + 3]);
    __syncwarp();
    const int col = k0 + h + piece * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + (lane >> 2);
      if (n0 + r < p.P && col < p.Q) {
        float4 w = *reinterpret_cast<const float4*>(at(r, piece));
        const size_t to = out + (size_t)(n0 + r) * p.Q + col;
        if (p.out32) {
          float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.out) + to);
          if (p.accumulate) {
            const float4 o = *d;
            w = make_float4(w.x + o.x, w.y + o.y, w.z + o.z, w.w + o.w);
          }
          *d = w;
        } else {
          uint2* d = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + to);
          const uint2 o = *d;
          float a[2], b[2];
          if (p.fp16) {
            Word<__half>::get(o.x, a);
            Word<__half>::get(o.y, b);
          } else {
            Word<__nv_bfloat16>::get(o.x, a);
            Word<__nv_bfloat16>::get(o.y, b);
          }
          *d = make_uint2(pack16(w.x + a[0], w.y + a[1], p.fp16), pack16(w.z + b[0], w.w + b[1], p.fp16));
        }
      }
    }
    __syncwarp();
  }
}

// KS: K blocks of a stage.  kPromote: see moe_linear's kernel.
template <Mode kMode, bool kPromote, int KS>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ Grouped p) {
  constexpr bool kAMN = kMode != kForward, kBMN = kMode == kDw;
  constexpr int kAStage = kRows * 128;  // bytes of a K block of A
  static_assert(kMode != kDw || KS == 1, "a tail is one K block");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ctrl = smem + kStageBudget;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tail = empty + kMaxStages;   // dw: this CTA's copies of a group's last block have landed
  uint64_t* fixed = tail + kMaxStages;   // dw, in the leader: the rows behind the end are zero in both CTAs
  uint64_t* tfull = fixed + kMaxStages;  // [2] accumulator complete
  uint64_t* tempty = tfull + 2;          // [2] accumulator read
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  char* bufs = reinterpret_cast<char*>(ctrl + kCtrlBytes);
  int* start = reinterpret_cast<int*>(bufs + kEpiWarps * kBufBytes);  // [E + 1] first sorted row of each group
  int* pre = start + kMaxE + 4;                                       // [E + 1] tiles of the groups before it
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int stages = p.stages, half_width = p.width / 2;
  const int b_stage = half_width * 128;  // bytes of a K block of B at most
  const int stage_bytes = KS * (kAStage + b_stage);
  const int half = (int)cluster_rank() & 1;
  const uint16_t pair_mask = 3;

  depend_launch();
  if (warp == 2 && elect_one()) {
    prefetch_tensormap(&tmA);
    prefetch_tensormap(&tmB);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&tail[s], 1);
      mbar_init(&fixed[s], 4);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kEpiWarps * 2);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_take<2>(tmem_slot);
  if (warp == 3) {
    int before = 0;
    for (int b = 0; b < p.E; b += 32) {
      const int e = b + lane;
      // (offsets out of order or range would be the caller's mistake; no row outside [0, S) is touched)
      const int first = e < p.E ? min(max(p.offsets[e], 0), p.S) : 0;
      const int end = e < p.E ? min(max(p.offsets[e + 1], 0), p.S) : 0;
      int n = (max(0, end - first) + p.width - 1) / p.width;
      const int own = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, n, off);
        if (lane >= off) n += v;
      }
      if (e < p.E) {
        start[e] = first;
        pre[e] = before + n - own;
      }
      if (e == p.E - 1) {
        start[p.E] = end;
        pre[p.E] = before + n;
      }
      before += __shfl_sync(0xffffffffu, n, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's barriers are set up
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  depend_wait();

  const int units = kMode == kDw ? p.E * p.tiles_p * p.tiles_q : p.tiles_p * pre[p.E];
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

  if (warp < kFirstEpi) {
    if (kPromote) setmaxnreg_dec<kLowRegs>();
    int stage = 0;
    uint32_t phase = 0;
    bool failed = false;
    auto advance = [&](int n) {  // n stages on
      stage += n;
      phase ^= (uint32_t)(stage / stages) & 1;
      stage %= stages;
    };
    if (warp == 0) {
      // ---------------------------------------------------------- TMA producer
      const uint64_t pol = policy_evict_normal();
      const uint32_t full0 = map_to_rank(smem_u32(full), 0);  // (both CTAs' copies complete there)
      uint32_t tailed = 0, tail_phase = 0;  // a bit a stage: its last use was a tail's; phase of its next tail
      for (int u = first; u < units; u += step) {
        const Unit t = unit_of<kMode>(p, start, pre, u);
        const int arow = (t.p * 2 + half) * kRows;
        const int boxes = kBMN ? half_width / 64 : (t.width / 2 + p.box - 1) / p.box;
        const int brow = kBMN ? t.q * p.width + half * half_width : t.row0 + half * (t.width / 2);
        const uint32_t bytes = KS * (kAStage + (kBMN ? b_stage : boxes * p.box * 128));
        if (elect_one()) {
          int st = stage;
          uint32_t ph = phase;
          for (int kb = 0; kb < t.stages; ++kb) {
            if (!lane_wait(&empty[st], ph ^ 1)) {
              failed = true;
              break;
            }
            uint8_t* sA = smem + st * stage_bytes;
            uint8_t* sB = sA + KS * kAStage;
            const bool last = kMode == kDw && kb == t.stages - 1 && t.rows % BK != 0;
            // a tail's copies complete in each CTA, where warps 2 and 3 wait for them
            const uint32_t bar = last ? smem_u32(&tail[st]) : full0 + st * 8;
            if (last) {
              mbar_arrive_expect_tx(&tail[st], bytes);
              if (half == 0) mbar_arrive(&full[st]);
              tailed |= 1u << st;
              tail_phase ^= 1u << st;
            } else {
              if (half == 0) mbar_arrive_expect_tx(&full[st], 2 * bytes);
              tailed &= ~(1u << st);
            }
            const int k = kMode == kDw ? t.row0 + kb * BK : kb * KS * BK;
            if constexpr (kMode == kForward) {
#pragma unroll
              for (int i = 0; i < KS; ++i)
                tma_load_pair_3d(sA + i * kAStage, &tmA, k + i * BK, arow, (int)t.e, bar, pol);
            } else if constexpr (kMode == kDx) {
#pragma unroll
              for (int g = 0; g < 2; ++g) tma_load_pair_3d(sA + g * KS * 8192, &tmA, arow + g * 64, k, (int)t.e, bar, pol);
            } else {
              auto load = [&](auto cg) {
#pragma unroll
                for (int g = 0; g < 2; ++g) tma_load<decltype(cg)::value>(sA + g * 8192, &tmA, arow + g * 64, k, bar, pol);
                for (int g = 0; g < boxes; ++g)
                  tma_load<decltype(cg)::value>(sB + g * 8192, &tmB, brow + g * 64, k, bar, pol);
              };
              if (last)
                load(std::integral_constant<int, 1>());
              else
                load(std::integral_constant<int, 2>());
            }
            if constexpr (!kBMN) {
#pragma unroll
              for (int i = 0; i < KS; ++i)
                for (int g = 0; g < boxes; ++g)
                  tma_load<2>(sB + i * b_stage + g * p.box * 128, &tmB, k + i * BK, brow + g * p.box, bar, pol);
            }
            if (++st == stages) {
              st = 0;
              ph ^= 1;
            }
          }
          if (failed) {
            // wait (bounded) for the copies still in flight: each stage's phase that the ring was in
            for (int i = 0; i < stages; ++i)
              if (tailed >> i & 1)
                mbar_wait(&tail[i], (tail_phase >> i & 1) ^ 1, false, 100000000ull);
              else if (half == 0)
                mbar_wait(&full[i], i < st ? ph : ph ^ 1, false, 100000000ull);
          }
        }
        __syncwarp();
        if ((failed = __any_sync(0xffffffffu, failed))) break;
        advance(t.stages);
      }
    } else if (warp == 1 && half == 0) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t a0 = smem_u32(smem), b0 = a0 + KS * kAStage;
      const uint32_t ad0 = desc_lo<kAMN, KS>(a0), bd0 = desc_lo<kBMN, KS>(b0);
      constexpr uint32_t kStepA = (kAMN ? 2048 : 32) >> 4, kStepB = (kBMN ? 2048 : 32) >> 4;  // 16 K elements on
      int acc = 0;
      uint32_t acc_phase = 0, fixed_phase = 0;  // fixed_phase: a bit a stage
      for (int u = first; u < units && !failed; u += step) {
        const Unit t = unit_of<kMode>(p, start, pre, u);
        const uint32_t idesc = p.idesc | (uint32_t)(t.width >> 3) << 17;
        const int chunk = kPromote ? p.chunk : t.stages;
        for (int kc = 0; kc < t.stages; kc += chunk) {
          const uint32_t d = tmem + acc * kAccCols;
          const int ke = min(t.stages, kc + chunk);
          uint32_t flip = 0;
          if (elect_one()) {
            int st = stage;
            uint32_t ph = phase;
            failed = !lane_wait(&tempty[acc], acc_phase ^ 1);
            tc_fence_after();
            for (int kb = kc; kb < ke && !failed; ++kb) {
              if (!lane_wait(&full[st], ph)) {
                failed = true;
                break;
              }
              if (kMode == kDw && kb == t.stages - 1 && t.rows % BK != 0) {
                if (!lane_wait_cluster(&fixed[st], fixed_phase >> st & 1)) {
                  failed = true;
                  break;
                }
                flip = 1u << st;
              }
              tc_fence_after();
              const uint32_t at = (uint32_t)(st * stage_bytes) >> 4;
#pragma unroll
              for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int kk = 0; kk < BK / 16; ++kk)
                  mma<2>(d, desc(ad0 + at + i * (kAMN ? 8192 >> 4 : kAStage >> 4) + kk * kStepA),
                         desc(bd0 + at + i * (kBMN ? 8192 >> 4 : b_stage >> 4) + kk * kStepB), idesc,
                         kb > kc || i > 0 || kk > 0);
              commit<2>(&empty[st], pair_mask);
              if (++st == stages) {
                st = 0;
                ph ^= 1;
              }
            }
            if (!failed) {
              commit<2>(&tfull[acc], pair_mask);
            } else {
              // a wait gave up: let the MMAs issued so far finish (bounded) before the tensor memory goes
              commit<2>(drain, pair_mask);
              mbar_wait(drain, 0, false, 100000000ull);
            }
          }
          __syncwarp();
          if ((failed = __any_sync(0xffffffffu, failed))) break;
          fixed_phase ^= __reduce_or_sync(0xffffffffu, flip);
          advance(ke - kc);
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1;
        }
      }
    } else if (kMode == kDw && warp >= 2) {
      // ---------------------------------------------------------- zeroes of dw's tails
      // warp 2 A's rows, warp 3 B's: a row of a box is 128 bytes whatever the swizzle, which stays within it
      const uint32_t fixed0 = map_to_rank(smem_u32(fixed), 0);
      uint32_t tail_phase = 0;
      for (int u = first; u < units; u += step) {
        const Unit t = unit_of<kMode>(p, start, pre, u);
        if (t.rows % BK != 0) {
          advance(t.stages - 1);
          if (!__all_sync(0xffffffffu, lane_wait(&tail[stage], tail_phase >> stage & 1))) break;
          tail_phase ^= 1u << stage;
          uint8_t* at = smem + stage * stage_bytes + (warp == 3 ? kAStage : 0);
          const int boxes = warp == 3 ? half_width / 64 : 2, from = t.rows % BK * 128;
          for (int b = 0; b < boxes; ++b)
            for (int i = from + lane * 16; i < 8192; i += 512)
              *reinterpret_cast<uint4*>(at + b * 8192 + i) = make_uint4(0, 0, 0, 0);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(fixed0 + stage * 8);
          advance(1);
        } else {
          advance(t.stages);
        }
      }
    }
    __syncwarp();
    // Every stage comes back before this CTA leaves: the commits of the pair's MMAs arrive on the barriers here.
    if (warp == 0 && elect_one() && !failed)
      for (int i = 0; i < stages && lane_wait<false>(&empty[stage], phase ^ 1); ++i)
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
  } else {
    // ------------------------------------------------------------ epilogue
    if (kPromote) setmaxnreg_inc<kHighRegs>();
    const int quarter = warp & 3;              // TMEM lanes this warp may access
    const int side = (warp - kFirstEpi) >> 2;  // every other 32 columns
    char* buf = bufs + (warp - kFirstEpi) * kBufBytes;
    const uint32_t tb = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t freed = map_to_rank(smem_u32(tempty), 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    auto release = [&]() {  // this warp is done with the accumulator
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(freed + acc * 8);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    };
    bool ok = true;
    for (int u = first; ok && u < units; u += step) {
      const Unit t = unit_of<kMode>(p, start, pre, u);
      const int n0 = (t.p * 2 + half) * kRows + quarter * 32;
      const int cols = n0 >= p.P ? 0 : kMode == kDw ? min(t.width, p.Q - t.q * p.width) : t.rows;
      auto take = [&](const float* v, int c) {
        if constexpr (kMode == kDw)
          store_grad32(p, buf, v, (size_t)t.e * p.P * p.Q, n0, t.q * p.width + c, lane);
        else
          store_rows32(p, buf, v, n0, t.row0 + c, t.rows - c, lane);
      };
      if (kMode == kDw && t.stages == 0) {  // an expert without rows
        if (!p.accumulate) {
          const float v[32] = {};
          for (int c = side * 32; c < cols; c += 64) take(v, c);
        }
        continue;
      }
      if constexpr (kPromote) {
        float sums[128] = {};
        for (int kc = 0; kc < t.stages; kc += p.chunk) {
          if (!(ok = __all_sync(0xffffffffu, lane_wait(&tfull[acc], acc_phase)))) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c * 64 + side * 32 < cols) {
#pragma unroll
              for (int h = 0; h < 32; h += 16) {
                float v[16];
                tmem_ld16(tb + acc * kAccCols + c * 64 + side * 32 + h, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) sums[c * 32 + h + i] += v[i];
              }
            }
          release();
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c * 64 + side * 32 < cols) take(sums + c * 32, c * 64 + side * 32);
      } else {
        if (!(ok = warp_wait(&tfull[acc], acc_phase))) break;
        tc_fence_after();
        for (int c = side * 32; c < cols; c += 64) {
          float v[32];
          tmem_ld32(tb + acc * kAccCols + c, v);
          tmem_ld_wait();
          take(v, c);
        }
        release();
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other uses its memory or barriers
  tc_fence_after();
  if (warp == 1) tmem_release<2>(tmem);
}

// ------------------------------------------------------------------ rows into sorted order
// to[p] = from[slots[p] / div] for the sorted rows p that belong to a group: a warp a row.
__global__ void __launch_bounds__(256)
    gather_rows_kernel(const uint4* __restrict__ from, const int32_t* __restrict__ slots,
                       const int32_t* __restrict__ offsets, int E, int S, int div, int nvec, uint4* __restrict__ to) {
  depend_launch();
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= S || row >= __ldg(offsets + E)) return;
  const int slot = __ldg(slots + row);
  uint4* d = to + (size_t)row * nvec;
  if (slot < 0 || slot >= S) {
    if (lane == 0) record_status((int)MOE_ERR_INVALID_ARG);
    for (int i = lane; i < nvec; i += 32) d[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const uint4* s = from + (size_t)(slot / div) * nvec;
  int i = lane;
  for (; i + 96 < nvec; i += 128) {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __ldg(s + i + j * 32);
#pragma unroll
    for (int j = 0; j < 4; ++j) d[i + j * 32] = v[j];
  }
  for (; i < nvec; i += 32) d[i] = __ldg(s + i);
}

// ------------------------------------------------------------------ host side
// A 16-bit tensor [outer][rows][inner] read in boxes of 64 inner elements x box rows of one matrix; outer 0: two
// dimensions.
bool make_map(CUtensorMap* m, const void* base, int fp16, long long inner, long long rows, long long outer, int box) {
  auto enc = get_encode();
  if (!enc) return false;
  const int rank = outer ? 3 : 2;
  cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)outer};
  cuuint64_t strides[2] = {(cuuint64_t)inner * 2, (cuuint64_t)inner * rows * 2};
  cuuint32_t boxes[3] = {64, (cuuint32_t)box, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base),
             dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <Mode kMode, bool kPromote, int KS>
cudaError_t launch(const CUtensorMap& ma, const CUtensorMap& mb, const Grouped& g, long long units, bool overlap,
                   cudaStream_t s) {
  auto kern = grouped_gemm_kernel<kMode, kPromote, KS>;
  if (kPromote) {
    // The epilogue's warps take registers that the first warpgroup gives back (setmaxnreg): a build with another
    // count than the split assumes would wait for them without an end, so it never launches.
    static std::atomic<bool> checked;
    if (!checked.load(std::memory_order_relaxed)) {
      cudaFuncAttributes fa;
      const cudaError_t e = cudaFuncGetAttributes(&fa, kern);
      if (e != cudaSuccess) return e;
      if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
      checked.store(true, std::memory_order_relaxed);
    }
  }
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = overlap_attr();
  cfg.attrs = attr;
  const long long pairs = num_sms() / 2;
  cfg.gridDim = dim3((unsigned)(2 * (units < pairs ? units : pairs)));
  cfg.numAttrs = overlap ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, ma, mb, g);
}
template <Mode kMode, bool kPromote>
cudaError_t launch(int ks, const CUtensorMap& ma, const CUtensorMap& mb, const Grouped& g, long long units, bool overlap,
                   cudaStream_t s) {
  if constexpr (kMode != kDw)
    if (ks == 2) return launch<kMode, kPromote, 2>(ma, mb, g, units, overlap, s);
  return launch<kMode, kPromote, 1>(ma, mb, g, units, overlap, s);
}

// One product.  a: the weights [E, N, K] (dw: dout, sorted), b: sorted rows.
template <Mode kMode>
moe_status_t run(const void* a, const void* b, const int32_t* offsets, const int32_t* slots, int S, int E, int N, int K,
                 int fp16, void* out, int out32, int accumulate, bool overlap, cudaStream_t s) {
  Grouped g = {};
  g.offsets = offsets;
  g.slots = slots;
  g.out = out;
  g.S = S;
  g.E = E;
  g.P = kMode == kDx ? K : N;
  g.Q = K;
  g.fp16 = fp16;
  g.out32 = out32;
  g.accumulate = accumulate;
  const int contraction = kMode == kForward ? K : kMode == kDx ? N : S;
  const long long mean = cdiv(S, E);
  int ks = 1;
  if (kMode == kDw) {
    g.width = K <= 128 ? 128 : 256;
  } else {
    g.width = S <= 32 ? 32 : mean <= 24 ? 64 : mean <= 48 ? 128 : 256;
    ks = g.width <= 128 ? 2 : 1;
  }
  g.box = g.width / 2 < 32 ? g.width / 2 : 32;
  g.tiles_p = cdiv(g.P, 2 * kRows);
  g.tiles_q = cdiv(g.Q, g.width);
  g.KB = cdiv(contraction, BK * ks);
  const int stage = ks * (kRows + g.width / 2) * 128;
  g.stages = kStageBudget / stage < kMaxStages ? kStageBudget / stage : kMaxStages;
  const int run = out32 ? kRunFP32 : fp16 ? kRunFP16 : kRunBF16;
  const bool promote = cdiv(contraction, BK) > run;
  g.chunk = run / ks;
  g.idesc = make_idesc(fp16 ? 0 : 1, 2 * kRows, 0) | (kMode != kForward ? 1u << 15 : 0) | (kMode == kDw ? 1u << 16 : 0);
  const long long units =
      kMode == kDw ? (long long)E * g.tiles_p * g.tiles_q : (long long)g.tiles_p * (S / g.width + (S < E ? S : E));
  if (units > 1073741823LL) return MOE_ERR_UNSUPPORTED;
  CUtensorMap ma, mb;
  bool ok;
  if (kMode == kDw)
    ok = make_map(&ma, a, fp16, N, S, 0, BK) && make_map(&mb, b, fp16, K, S, 0, BK);
  else
    ok = make_map(&ma, a, fp16, K, N, E, kMode == kForward ? kRows : BK * ks) &&
         make_map(&mb, b, fp16, kMode == kForward ? K : N, S, 0, g.box);
  if (!ok) return MOE_ERR_CUDA;
  const cudaError_t err = promote ? launch<kMode, true>(ks, ma, mb, g, units, overlap, s)
                                  : launch<kMode, false>(ks, ma, mb, g, units, overlap, s);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Rows in `order` -> sorted rows at `to` (the caller's where they are sorted already).
const void* sorted_rows(const void* from, int order, const int32_t* offsets, const int32_t* slots, int S, int E, int cols,
                        int top_k, void* to, cudaStream_t s) {
  if (order == MOE_ROWS_SORTED) return from;
  gather_rows_kernel<<<cdiv(S, 8), 256, 0, s>>>(static_cast<const uint4*>(from), slots, offsets, E, S,
                                                order == MOE_ROWS_TOKEN ? top_k : 1, cols / 8, static_cast<uint4*>(to));
  return to;
}

size_t rows_bytes(long long S, long long cols, int order) {
  return order == MOE_ROWS_SORTED ? 0 : ((size_t)S * cols * 2 + 255) / 256 * 256;
}

bool order_ok(int order, const int32_t* slots, int S, int top_k, bool token) {
  if (order < MOE_ROWS_SORTED || order > (token ? MOE_ROWS_TOKEN : MOE_ROWS_SLOT)) return false;
  return order == MOE_ROWS_SORTED || (slots && (order != MOE_ROWS_TOKEN || S % top_k == 0));
}

moe_status_t check_sizes(int S, int E, int N, int K, int top_k, moe_dtype_t dtype) {
  MOE_CHECK_ARG(S >= 0 && S <= (1 << 30) && E >= 1 && E <= kMaxE && top_k >= 1);
  MOE_CHECK_ARG(N >= 8 && N % 8 == 0 && N <= (1 << 21) && K >= 8 && K % 8 == 0 && K <= (1 << 21));
  return dtype == MOE_DT_BF16 || dtype == MOE_DT_FP16 ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

}  // namespace

MOE_DEFINE_STATUS_READER(grouped_status)

}  // namespace moe

using namespace moe;

extern "C" size_t moe_grouped_linear_workspace_size(int S, int E, int N, int K, int x_rows) {
  if (S <= 0 || E <= 0 || N <= 0 || K <= 0) return 0;
  return rows_bytes(S, K, x_rows);
}

extern "C" moe_status_t moe_grouped_linear(const void* x, int x_rows, const void* w, const int32_t* expert_offsets,
                                           const int32_t* sorted_slot, int S, int E, int N, int K, int top_k,
                                           moe_dtype_t dtype, void* out, int out_rows, void* ws, size_t ws_bytes,
                                           moe_stream_t stream) {
  const moe_status_t st = check_sizes(S, E, N, K, top_k, dtype);
  if (st != MOE_OK) return st;
  if (S == 0) return MOE_OK;
  MOE_CHECK_ARG(x && w && expert_offsets && out);
  MOE_CHECK_ARG(order_ok(x_rows, sorted_slot, S, top_k, true) && order_ok(out_rows, sorted_slot, S, top_k, false));
  MOE_CHECK_ARG(aligned16(x) && aligned16(w) && aligned16(expert_offsets) && aligned16(sorted_slot) && aligned16(out) &&
                aligned16(ws));
  const size_t need = rows_bytes(S, K, x_rows);
  if (need && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const void* xs = sorted_rows(x, x_rows, expert_offsets, sorted_slot, S, E, K, top_k, ws, s);
  const moe_status_t got =
      run<kForward>(w, xs, expert_offsets, out_rows == MOE_ROWS_SLOT ? sorted_slot : nullptr, S, E, N, K,
                    dtype == MOE_DT_FP16, out, 0, 0, xs != x, s);
  return got == MOE_OK ? launch_status() : got;
}

extern "C" size_t moe_grouped_linear_backward_workspace_size(int S, int E, int N, int K, int dout_rows, int x_rows) {
  if (S <= 0 || E <= 0 || N <= 0 || K <= 0) return 0;
  return rows_bytes(S, N, dout_rows) + rows_bytes(S, K, x_rows);
}

extern "C" moe_status_t moe_grouped_linear_backward(const void* dout, int dout_rows, const void* x, int x_rows,
                                                    const void* w, const int32_t* expert_offsets,
                                                    const int32_t* sorted_slot, int S, int E, int N, int K, int top_k,
                                                    moe_dtype_t dtype, void* dx, int dx_rows, void* dw,
                                                    moe_dtype_t dw_dtype, int accumulate, void* ws, size_t ws_bytes,
                                                    moe_stream_t stream) {
  moe_status_t st = check_sizes(S, E, N, K, top_k, dtype);
  if (st != MOE_OK) return st;
  if (dw_dtype != dtype && dw_dtype != MOE_DT_FP32) return MOE_ERR_UNSUPPORTED;
  MOE_CHECK_ARG(dx || dw);
  MOE_CHECK_ARG(aligned16(dx) && aligned16(dw));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int out32 = dw_dtype == MOE_DT_FP32;
  if (S == 0) {
    if (dw && !accumulate && cudaMemsetAsync(dw, 0, (size_t)E * N * K * (out32 ? 4 : 2), s) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  MOE_CHECK_ARG(dout && expert_offsets && (!dx || w) && (!dw || x));
  MOE_CHECK_ARG(order_ok(dout_rows, sorted_slot, S, top_k, true) && order_ok(x_rows, sorted_slot, S, top_k, true) &&
                order_ok(dx_rows, sorted_slot, S, top_k, false));
  MOE_CHECK_ARG(aligned16(dout) && aligned16(x) && aligned16(w) && aligned16(expert_offsets) && aligned16(sorted_slot) &&
                aligned16(ws));
  const size_t first = rows_bytes(S, N, dout_rows), need = first + (dw ? rows_bytes(S, K, x_rows) : 0);
  if (need && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  const int fp16 = dtype == MOE_DT_FP16;
  const void* d = sorted_rows(dout, dout_rows, expert_offsets, sorted_slot, S, E, N, top_k, ws, s);
  const void* xs =
      dw ? sorted_rows(x, x_rows, expert_offsets, sorted_slot, S, E, K, top_k, static_cast<uint8_t*>(ws) + first, s) : x;
  bool overlap = d != dout || xs != x;
  if (dx) {
    st = run<kDx>(w, d, expert_offsets, dx_rows == MOE_ROWS_SLOT ? sorted_slot : nullptr, S, E, N, K, fp16, dx, 0, 0,
                  overlap, s);
    if (st != MOE_OK) return st;
    overlap = true;
  }
  if (dw) {
    st = run<kDw>(d, xs, expert_offsets, nullptr, S, E, N, K, fp16, dw, out32, accumulate != 0, overlap, s);
    if (st != MOE_OK) return st;
  }
  return launch_status();
}
