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
// token's experts read their weights once over narrow tiles.  dw has no ragged side but its contraction: a small
// kernel makes tensor maps that end with each group, so that the copies of a group's last rows bring zeros
// for what lies behind them.  (Zeroing those rows in shared memory between copy and MMAs stalled the K loop some 2500
// clocks a tile: both gradients of 4096 x 14336 over groups of 1024 rows 1338 us, like this 1207.)
//
// Where there are few tiles, forward and dx split the contraction over two or four pairs of a cluster: each leaves its
// fp32 partial tile in its own shared memory, and after one cluster barrier every pair adds its share of the columns
// over distributed shared memory, in rank order.
//
// Persistent, warp-specialised, pairs of CTAs: warps 0 and 2 copy stages of K blocks of A and of B by TMA (one warp for
// both was busy 65 % of its time where K loops are short), warp 1 issues the MMAs, warps 4-11 run the epilogue from one of two accumulators in tensor memory while the
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
constexpr int kCtrlBytes = 512;
constexpr int kSmemMost = 232448;
enum Mode { kForward, kDx, kDw };
// Shared memory: the stages (as many as fit), a buffer for each epilogue warp, barriers, the groups' table.
constexpr int buf_bytes(Mode m) { return m == kDw ? 4096 : 2048; }
constexpr int table_bytes(Mode m, int E) { return (m == kDw ? 1 : 2) * ((E + 4) & ~3) * 4; }
constexpr int smem_bytes(Mode m, int E, int stages, int stage) {
  return 1024 + stages * stage + kEpiWarps * buf_bytes(m) + kCtrlBytes + table_bytes(m, E);
}
// K blocks of a sum in tensor memory, whose additions truncate, by the output's type; longer ones are added up in
// fp32 registers with rounding (kPromote), as moe_linear's are
constexpr int kRunFP32 = 8, kRunFP16 = 128, kRunBF16 = 256;
// stages that splitting a tile's contraction has to save to be worth its cluster barrier and joining: not split / split, 306
// rows of 9 experts, 256 over 9512 37 / 19 us; 2 of 8, 1024 over 4096 13 / 10.4; 512 of 2, 512 over 2048 16 / 13; 17 of 4,
// 1472 over 3168 (saves 19) 11.9 / 13.0
constexpr int kSplitGain = 20;
constexpr int kLaunchRegs = 168, kLowRegs = 40, kHighRegs = 232;
static_assert(128 * kLowRegs + 256 * kHighRegs == kThreads * kLaunchRegs, "register split must balance");
static_assert((2 * kMaxStages + 5) * 8 + 4 <= 256 && 256 + 32 * 4 <= kCtrlBytes && smem_bytes(kForward, kMaxE, 6, 32768) <= kSmemMost && smem_bytes(kDw, kMaxE, 5, 32768) <= kSmemMost, "shared memory layout");

// Bad offsets and slots are kept apart from the status word: a wait gives up when that is set, and they are no reason to.
static __device__ int g_invalid = 0;
__device__ __forceinline__ void record_invalid() { atomicExch(&g_invalid, (int)MOE_ERR_INVALID_ARG); }

struct Grouped {
  const CUtensorMap* ends;         // dw: maps of dout and x that end with each group
  const int32_t *offsets, *slots;  // slots: NULL where no order needs them
  int to_slots;                    // rows of out are the slots of the sorted rows (else the sorted rows)
  const int32_t* from;             // forward, small groups: B's rows are those of slots / from_div, fetched one by one
  int from_div;
  void* out;
  int S, E;
  int P, Q;              // rows of A's tensor (forward N, dx K, dw N); dw: columns of B's (K)
  int KB;                // stages of the contraction (dw: by the group's rows)
  int splits;            // pairs of a cluster that share a tile's (forward, dx; more than one: a tile a cluster)
  int tiles_p, tiles_q;  // of 256 rows of A; dw: of `width` columns
  int per;               // dw: tiles of an expert
  unsigned long long per_inverse;  // floor(2^64 / per) + 1: the high word of u times it is u / per
  int width, log2_width; // columns of a tile at most (a power of two)
  int stages, chunk;     // chunk: stages added up in the tensor memory (kPromote)
  int fp16, out32, accumulate;
  int wide_a, wide_b;    // dw: an operand's 128 columns are one copy (see make_rows_map)
  uint32_t idesc;        // but for the columns
};

// Forward, dx: B's tensor in boxes of 16, 32, .. rows, one for each half tile there can be, so that a K block of B is
// one copy whatever the tile (in boxes of 32 rows the copies' issue bounded the K loop).
struct Maps {
  CUtensorMap b[8];
};

struct Unit {
  int p, q;        // tile of A; dw: of B
  int row0, rows;  // sorted rows: of the tile (forward, dx), of the group (dw)
  int width;       // columns of the tile
  int stage0, stages;  // of its contraction, this pair's
  long long e;
};

// a / d: exact below 2^20 by way of the reciprocal, whose error there is a quarter of the distance to the next quotient
// (an integer division would be most of a tile's bookkeeping, which short K loops do not hide).
__device__ __forceinline__ int quotient(int a, int d) {
  if (d == 1) return a;
  return a < (1 << 20) ? (int)(((float)a + 0.5f) * __frcp_rn((float)d)) : a / d;
}
// Blocks of up to 8 tile columns run through all tile rows (dw: the other way round), so that the pairs that work at
// the same time share both operands in L2.
constexpr int kRaster = 8;
__device__ __forceinline__ void raster(int in, int many, int other, int& a, int& b) {
  int first = 0, n = many;
  if (many > kRaster) {
    const int blocks = (many + kRaster - 1) / kRaster, r = quotient(many + blocks - 1, blocks), g = quotient(in, r * other);
    first = g * r;
    in -= first * other;
    n = min(r, many - first);
  }
  b = quotient(in, n);
  a = first + in - b * n;
}
// The tile of the unit u.  For a whole warp.
template <Mode kMode, bool kSplit>
__device__ __forceinline__ Unit unit_of(const Grouped& p, const int* start, const int* pre, int u, int lane, int split) {
  Unit t;
  if constexpr (kMode == kDw) {
    const int e = p.per == 1 ? u : (int)__umul64hi((unsigned long long)u, p.per_inverse);
    raster(u - e * p.per, p.tiles_p, p.tiles_q, t.p, t.q);
    t.e = e;
    t.row0 = start[e];
    t.rows = max(0, start[e + 1] - t.row0);
    t.width = p.width;
    t.stage0 = 0;
    t.stages = (t.rows + BK - 1) / BK;
  } else {
    int e = 0, span = p.E;  // the last e with pre[e] <= u is in [e, e + span)
    while (span > 1) {
      const int stride = (span + 31) >> 5, i = lane * stride;
      const int last = __popc(__ballot_sync(0xffffffffu, i < span && pre[min(e + i, p.E)] <= u)) - 1;
      e += last * stride;
      span = min(stride, span - last * stride);
    }
    const int rows = start[e + 1] - start[e], n = (rows + p.width - 1) >> p.log2_width;
    raster(u - pre[e], n, p.tiles_p, t.q, t.p);
    t.e = e;
    // the group's rows dealt evenly over its tiles (that many are needed, so none is empty)
    t.width = (quotient(rows + n - 1, n) + 31) & ~31;
    t.row0 = start[e] + t.q * t.width;
    t.rows = min(t.width, rows - t.q * t.width);
    t.stage0 = kSplit ? p.KB * split / p.splits : 0;
    t.stages = kSplit ? p.KB * (split + 1) / p.splits - t.stage0 : p.KB;
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
// Four rows of a tensor (a box is one row of 64 elements).
__device__ __forceinline__ void tma_gather4_pair(void* smem_dst, const CUtensorMap* map, int x, int4 rows, uint32_t bar,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w), "r"(bar), "l"(policy)
      : "memory");
}
// A tensor map in global memory that an earlier kernel wrote.
__device__ __forceinline__ void acquire_map(const CUtensorMap* map) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack16(float a, float b, int fp16) {
  const float v[2] = {a, b};
  return fp16 ? Word<__half>::put(v) : Word<__nv_bfloat16>::put(v);
}

// Without order: the accumulator's values are in registers (tcgen05.wait::ld), and a release would wait for the
// thread's stores to global memory too (over a microsecond).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// 32 rows of A (lanes, from n0) x 32 sorted rows into out, 16 bits (w: sorted rows 2 i and 2 i + 1 in word i),
// transposed through the warp's buffer: lanes pair up so that a word holds two neighbouring columns of out.  to: of
// each sorted row (lane) its row of out, below 0 where it has none.
__device__ __forceinline__ void store_rows32(const Grouped& p, char* buf, const uint32_t (&w)[16], int n0, int to, int lane) {
  uint32_t* words = reinterpret_cast<uint32_t*>(buf);
  const bool odd = lane & 1;
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    const uint32_t mine = w[c], other = __shfl_xor_sync(0xffffffffu, mine, 1);
    words[(2 * c + odd) * 16 + (lane >> 1)] = odd ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x5410);
  }
  __syncwarp();
  const int piece = lane & 3, col = n0 + piece * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = i * 8 + (lane >> 2), row = __shfl_sync(0xffffffffu, to, c);
    const uint4 v = *reinterpret_cast<const uint4*>(buf + c * 64 + piece * 16);
    if (row >= 0 && col < p.P) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (size_t)row * p.P + col) = v;
  }
  __syncwarp();
}

// ---- a weight gradient: 32 rows x 128 bytes at a time, by TMA from the warp's buffer (128-byte swizzle; what lies
// behind the matrix is clipped)
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* smem_src, int x, int y, int z, bool add) {
  if (add)
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(smem_u32(smem_src))
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(smem_u32(smem_src))
                 : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The thread's stores have read their buffers.
__device__ __forceinline__ void tma_store_wait() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

__device__ __forceinline__ char* grad_at(char* buf, int row, int piece) { return buf + row * 128 + ((piece ^ (row & 7)) << 4); }

// 32 words of a row in each lane.
__device__ __forceinline__ void store_grad(const CUtensorMap* map, char* buf, const uint32_t* w, int n0, int k0, int e, bool add,
                                           int lane) {
  if (lane == 0) tma_store_wait();
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint4*>(grad_at(buf, lane, i)) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  fence_async_smem();
  __syncwarp();
  if (lane == 0) tma_store_3d(map, buf, k0, n0, e, add);
}

// 32 x 32 sums added to 16-bit gradients, in fp32, rounded once.
__device__ __forceinline__ void add_grad16(const Grouped& p, char* buf, const float* v, int n0, int k0, size_t out, int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<float4*>(grad_at(buf, lane, i)) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  __syncwarp();
  const int piece = lane & 7, col = k0 + piece * 4;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 4 + (lane >> 3);
    if (n0 + r < p.P && col < p.Q) {
      const float4 w = *reinterpret_cast<const float4*>(grad_at(buf, r, piece));
      uint2* d = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + out + (size_t)(n0 + r) * p.Q + col);
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
  __syncwarp();
}

// KS: K blocks of a stage.  kPromote: see moe_linear's kernel.  kSplit: p.splits pairs share a tile's contraction (in the
// other kernels its branches cost 2 % of short tiles).
template <Mode kMode, bool kPromote, int KS, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ Maps maps,
                        const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ Grouped p) {
  constexpr bool kAMN = kMode != kForward, kBMN = kMode == kDw;
  constexpr int kAStage = kRows * 128;  // bytes of a K block of A
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int stages = p.stages, half_width = p.width / 2;
  const int b_stage = half_width * 128;  // bytes of a K block of B at most
  const int stage_bytes = KS * (kAStage + b_stage);
  char* bufs = reinterpret_cast<char*>(smem + stages * stage_bytes);
  uint8_t* ctrl = reinterpret_cast<uint8_t*>(bufs + kEpiWarps * buf_bytes(kMode));
  uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;  // [2] accumulator complete
  uint64_t* tempty = tfull + 2;          // [2] accumulator read
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* rows4 = reinterpret_cast<int*>(ctrl + 256);  // B's rows of the producer's tile (p.from)
  int* start = reinterpret_cast<int*>(ctrl + kCtrlBytes);  // [E + 1] first sorted row of each group
  int* pre = start + ((p.E + 4) & ~3);                     // [E + 1] units of the groups before it (not dw's)
  // cluster: the pairs that share a tile; the even CTA of a pair issues its MMAs
  const int rank = (int)cluster_rank(), half = rank & 1, split = rank >> 1;
  const uint32_t leader = rank - half;
  const uint16_t pair_mask = (uint16_t)(3u << leader);

  depend_launch();
  if (warp == 2 && elect_one()) {
    if (kMode == kDw) {
      prefetch_tensormap(&tmOut);
    } else {
      prefetch_tensormap(&tmA);
      for (int i = 0; i < (p.from ? 1 : p.width / 32); ++i) prefetch_tensormap(&maps.b[i]);
    }
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kEpiWarps * 2);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  __syncwarp();
  // The pair meets twice: here, with its barriers set up, and (half a microsecond later, under the rest) below.
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (warp == 1) tmem_take<2>(tmem_slot);
  if (warp == 3) {  // the groups' rows and tiles
    int before = 0;
    for (int b = 0; b < p.E; b += 128) {
      int first[4], end[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = b + j * 32 + lane;
        first[j] = e < p.E ? __ldg(p.offsets + e) : 0;
        end[j] = e < p.E ? __ldg(p.offsets + e + 1) : 0;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = b + j * 32 + lane;
        if (b + j * 32 >= p.E) break;
        // (the caller's mistake; no row outside [0, S) is touched)
        if (first[j] < 0 || first[j] > end[j] || end[j] > p.S) record_invalid();
        first[j] = min(max(first[j], 0), p.S);
        end[j] = min(max(end[j], 0), p.S);
        int n = p.tiles_p * ((max(0, end[j] - first[j]) + p.width - 1) >> p.log2_width);
        if (e < p.E) start[e] = first[j];
        if (e == p.E - 1) start[p.E] = end[j];
        if (kMode == kDw) continue;
        const int own = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, n, off);
          if (lane >= off) n += v;
        }
        if (e < p.E) pre[e] = before + n - own;
        before += __shfl_sync(0xffffffffu, n, 31);
      }
    }
    if (kMode != kDw && lane == 0) pre[p.E] = before;
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int units = kMode == kDw ? p.E * p.per : pre[p.E];
  const int splits = kSplit ? p.splits : 1;
  const int first = blockIdx.x / (2 * splits), step = kSplit ? units : gridDim.x >> 1;

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
      // ---------------------------------------------------------- TMA producer of A
      const uint64_t pol = policy_evict_normal();
      const uint32_t full0 = map_to_rank(smem_u32(full), leader);  // (both CTAs' copies complete there)
      long long seen = -1;  // dw: the group whose map was acquired
      if (kMode == kDw) depend_wait();  // (the weights are the caller's and wait for nothing in this call)
      for (int u = first; u < units; u += step) {
        const Unit t = unit_of<kMode, kSplit>(p, start, pre, u, lane, split);
        const int arow = (t.p * 2 + half) * kRows;
        const CUtensorMap* mA = kMode == kDw ? p.ends + 2 * t.e : &tmA;
        uint32_t bytes = 2 * KS * (kAStage + (kBMN ? b_stage : t.width / 2 * 128));  // of a stage, both CTAs', A and B
        if (kMode == kForward && p.from) {
          const int n = t.width / 2;
          bytes = KS * (2 * kAStage + ((min(t.rows, n) + 3) / 4 + (max(0, t.rows - n) + 3) / 4) * 512);
        }
        if (elect_one()) {
          if (kMode == kDw && seen != t.e && t.stages) acquire_map(mA);
          int st = stage;
          uint32_t ph = phase;
          for (int kb = 0; kb < t.stages; ++kb) {
            if (!lane_wait(&empty[st], ph ^ 1)) {
              failed = true;
              break;
            }
            uint8_t* sA = smem + st * stage_bytes;
            const uint32_t bar = full0 + st * 8;
            if (half == 0) mbar_arrive_expect_tx(&full[st], bytes);
            const int k = kMode == kDw ? t.row0 + kb * BK : (t.stage0 + kb) * KS * BK;
            if constexpr (kMode == kForward) {
#pragma unroll
              for (int i = 0; i < KS; ++i)
                tma_load_pair_3d(sA + i * kAStage, mA, k + i * BK, arow, (int)t.e, bar, pol);
            } else if (kMode == kDw && p.wide_a) {
              tma_load_pair_3d(sA, mA, 0, k, arow / 64, bar, pol);
            } else {
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                if (kMode == kDx)
                  tma_load_pair_3d(sA + g * KS * 8192, mA, arow + g * 64, k, (int)t.e, bar, pol);
                else
                  tma_load<2>(sA + g * 8192, mA, arow + g * 64, k, bar, pol);
              }
            }
            if (++st == stages) {
              st = 0;
              ph ^= 1;
            }
          }
          if (failed) {
            // wait (bounded) for the copies still in flight, B's too: each stage's phase that the ring was in
            if (half == 0)
              for (int i = 0; i < stages; ++i) mbar_wait(&full[i], i < st ? ph : ph ^ 1, false, 100000000ull);
          }
        }
        __syncwarp();
        if ((failed = __any_sync(0xffffffffu, failed))) break;
        advance(t.stages);
        seen = t.stages ? t.e : seen;
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------- TMA producer of B
      const uint64_t pol = policy_evict_normal();
      const uint32_t full0 = map_to_rank(smem_u32(full), leader);
      long long seen = -1;
      depend_wait();  // (rows put in order by an earlier kernel of this call)
      for (int u = first; u < units; u += step) {
        const Unit t = unit_of<kMode, kSplit>(p, start, pre, u, lane, split);
        const int brow = kBMN ? t.q * p.width + half * half_width : t.row0 + half * (t.width / 2);
        const CUtensorMap* mB =
            kMode == kDw ? p.ends + 2 * t.e + 1 : &maps.b[kMode == kForward && p.from ? 0 : t.width / 32 - 1];
        int fours = 0;  // p.from: this CTA's rows, by four
        if (kMode == kForward && p.from) {
          // (the columns of the tile that have no row keep what the stage held; nobody looks at their sums)
          const int n = t.width / 2, have = max(0, min(t.rows - half * n, n));
          fours = (have + 3) / 4;
          __syncwarp();
          int slot = have ? __ldg(p.from + t.row0 + half * n + min(lane, have - 1)) : 0;
          if (slot < 0 || slot >= p.S) {
            record_invalid();
            slot = 0;
          }
          rows4[lane] = slot / p.from_div;
          __syncwarp();
        }
        if (elect_one()) {
          if (kMode == kDw && seen != t.e && t.stages) acquire_map(mB);
          int st = stage;
          uint32_t ph = phase;
          for (int kb = 0; kb < t.stages; ++kb) {
            if (!lane_wait(&empty[st], ph ^ 1)) {
              failed = true;
              break;
            }
            uint8_t* sB = smem + st * stage_bytes + KS * kAStage;
            const uint32_t bar = full0 + st * 8;
            const int k = kMode == kDw ? t.row0 + kb * BK : (t.stage0 + kb) * KS * BK;
            if (kMode == kForward && p.from) {
              for (int g = 0; g < fours; ++g) {
                const int4 rows = reinterpret_cast<const int4*>(rows4)[g];
#pragma unroll
                for (int i = 0; i < KS; ++i) tma_gather4_pair(sB + i * b_stage + g * 512, mB, k + i * BK, rows, bar, pol);
              }
            } else if constexpr (!kBMN) {
#pragma unroll
              for (int i = 0; i < KS; ++i) tma_load<2>(sB + i * b_stage, mB, k + i * BK, brow, bar, pol);
            } else if (p.wide_b) {
              tma_load_pair_3d(sB, mB, 0, k, brow / 64, bar, pol);
            } else {
              for (int g = 0; g < half_width / 64; ++g) tma_load<2>(sB + g * 8192, mB, brow + g * 64, k, bar, pol);
            }
            if (++st == stages) {
              st = 0;
              ph ^= 1;
            }
          }
        }
        __syncwarp();
        if ((failed = __any_sync(0xffffffffu, failed))) break;
        advance(t.stages);
        seen = t.stages ? t.e : seen;
      }
    } else if (warp == 1 && half == 0) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t a0 = smem_u32(smem), b0 = a0 + KS * kAStage;
      const uint32_t ad0 = desc_lo<kAMN, KS>(a0), bd0 = desc_lo<kBMN, KS>(b0);
      constexpr uint32_t kStepA = (kAMN ? 2048 : 32) >> 4, kStepB = (kBMN ? 2048 : 32) >> 4;  // 16 K elements on
      int acc = 0;
      uint32_t acc_phase = 0;
      for (int u = first; u < units && !failed; u += step) {
        const Unit t = unit_of<kMode, kSplit>(p, start, pre, u, lane, split);
        const uint32_t idesc = p.idesc | (uint32_t)(t.width >> 3) << 17;
        const int chunk = kPromote ? p.chunk : t.stages;
        for (int kc = 0; kc < t.stages; kc += chunk) {
          const uint32_t d = tmem + acc * kAccCols;
          const int ke = min(t.stages, kc + chunk);
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
          advance(ke - kc);
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1;
        }
      }
    }
    __syncwarp();
    if (kSplit) cluster_sync();  // (the partial tiles are in shared memory)
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
    const int side = (warp - kFirstEpi) >> 2;  // forward, dx: every other 32 columns; dw: half of them
    char* buf = bufs + (warp - kFirstEpi) * buf_bytes(kMode);
    const uint32_t tb = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t freed = map_to_rank(smem_u32(tempty), leader);
    int acc = 0;
    uint32_t acc_phase = 0;
    auto release = [&]() {  // this warp is done with the accumulator
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(freed + acc * 8);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    };
    bool ok = true;
    // first column of the c-th 32 columns of this warp, in the tile
    auto at = [&](int c) { return kMode == kDw ? side * (p.width / 2) + c * 32 : c * 64 + side * 32; };
    // Rows of out of a tile's columns (see store_rows32).  (Asked for a tile ahead: their latency would be a good part
    // of a short tile's time.)
    auto row_of = [&](const Unit& t, int col) {
      const int row = col < t.rows ? t.row0 + col : -1;
      if (!p.slots || row < 0) return row;
      const int slot = __ldg(p.slots + row);
      const bool bad = slot < 0 || slot >= p.S;
      if (bad) record_invalid();
      return bad ? -1 : p.to_slots ? slot : row;
    };
    auto rows_of = [&](const Unit& t, int (&to)[4]) {
#pragma unroll
      for (int c = 0; c < 4; ++c) to[c] = row_of(t, at(c) + lane);
    };
    // A split tile's sums, by columns: a column's 128 rows are neighbours (this CTA's stages: every copy has landed and
    // every MMA has read it when the accumulator is complete).
    float* part = reinterpret_cast<float*>(smem) + quarter * 32 + lane;
    Unit t = {};
    int to[4] = {};
    if (first < units) {
      t = unit_of<kMode, kSplit>(p, start, pre, first, lane, split);
      if (kMode != kDw) rows_of(t, to);
    }
    for (int u = first; u < units; u += step) {
      const int n0 = (t.p * 2 + half) * kRows + quarter * 32;
      // columns of the tile that are of use
      const int cols = n0 >= p.P ? 0 : kMode == kDw ? min((side + 1) * (p.width / 2), p.Q - t.q * p.width) : t.rows;
      uint32_t words[kPromote ? 1 : 4][16] = {};
      float sums[kPromote ? 128 : 1] = {};
      if (kMode != kDw || t.stages > 0) {
        if constexpr (kPromote) {
          for (int kc = 0; kc < t.stages; kc += p.chunk) {
            if (!(ok = __all_sync(0xffffffffu, lane_wait(&tfull[acc], acc_phase)))) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (at(c) < cols) {
#pragma unroll
                for (int h = 0; h < 32; h += 16) {
                  float v[16];
                  tmem_ld16(tb + acc * kAccCols + at(c) + h, v);
                  tmem_ld_wait();
#pragma unroll
                  for (int i = 0; i < 16; ++i) sums[c * 32 + h + i] += v[i];
                }
              }
            release();
          }
          if (!ok) break;
        } else {
          if (!(ok = warp_wait(&tfull[acc], acc_phase))) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (at(c) < cols) {
              float v[32];
              tmem_ld32(tb + acc * kAccCols + at(c), v);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) words[c][i] = pack16(v[2 * i], v[2 * i + 1], p.fp16);
              if (kSplit) {
#pragma unroll
                for (int i = 0; i < 32; ++i) part[(at(c) + i) * kRows] = v[i];
              }
            }
          release();
        }
      }
      Unit next = {};
      int next_to[4] = {};
      if (u + step < units) {
        next = unit_of<kMode, kSplit>(p, start, pre, u + step, lane, split);
        if (kMode != kDw) rows_of(next, next_to);
      }
      // the c-th 32 columns in 16 bits, two to a word
      auto packed = [&](int c, uint32_t* w) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if constexpr (kPromote)
            w[i] = pack16(sums[c * 32 + 2 * i], sums[c * 32 + 2 * i + 1], p.fp16);
          else
            w[i] = words[c][i];
        }
      };
      if (kSplit) {  // (joined below)
        if constexpr (kPromote) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (at(c) < cols) {
#pragma unroll
              for (int i = 0; i < 32; ++i) part[(at(c) + i) * kRows] = sums[c * 32 + i];
            }
        }
        break;
      }
      if constexpr (kMode != kDw) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (at(c) < cols) {
            uint32_t w[16];
            packed(c, w);
            store_rows32(p, buf, w, n0, to[c], lane);
          }
      } else {
        const int k0 = t.q * p.width;
        if (t.stages == 0) {
          // An expert without rows: its gradient is zeros in one piece, of which this unit and warp take a share (by
          // tiles, rows that start on no multiple of 32 bytes took twice the time).
          if (!p.accumulate) {
            const long long all = (long long)p.P * p.Q / (p.out32 ? 4 : 8);  // 16-byte vectors
            const int shares = p.per * 2 * kEpiWarps, mine = ((u - (int)t.e * p.per) * 2 + half) * kEpiWarps + warp - kFirstEpi;
            const long long each = ((all + shares - 1) / shares + 7) & ~7ll, end = min(all, (mine + 1) * each);
            uint4* d = static_cast<uint4*>(p.out) + t.e * all;
            for (long long i = mine * each + lane; i < end; i += 32) d[i] = make_uint4(0, 0, 0, 0);
          }
        } else if (!(kPromote && (p.out32 || p.accumulate))) {
#pragma unroll
          for (int c = 0; c < 4; c += 2)
            if (at(c) < cols) {
              uint32_t w[32];
              packed(c, w);
              packed(c + 1, w + 16);
              store_grad(&tmOut, buf, w, n0, k0 + at(c), (int)t.e, false, lane);
            }
        } else if constexpr (kPromote) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (at(c) < cols) {
              if (p.out32)
                store_grad(&tmOut, buf, reinterpret_cast<const uint32_t*>(sums + c * 32), n0, k0 + at(c), (int)t.e,
                           p.accumulate, lane);
              else
                add_grad16(p, buf, sums + c * 32, n0, k0 + at(c), (size_t)t.e * p.P * p.Q, lane);
            }
        }
      }
      t = next;
#pragma unroll
      for (int c = 0; c < 4; ++c) to[c] = next_to[c];
    }
    if (kMode == kDw && lane == 0) tma_store_wait();
    if (kSplit) {
      __syncwarp();
      cluster_sync();  // every pair's partial tile is in its shared memory
      const int n0 = (t.p * 2 + half) * kRows + quarter * 32, cols = first < units && n0 < p.P ? t.rows : 0;
      const uint32_t mine = smem_u32(part);
      // (a wait that gave up, here or in another CTA, leaves wrong values, and is recorded)
      for (int c = (side * splits + split) * 32; c < cols; c += 64 * splits) {
        const int row = row_of(t, c + lane);
        uint32_t w[16];
#pragma unroll
        for (int h = 0; h < 32; h += 8) {
          float z[8] = {};
          for (int s = 0; s < splits; ++s) {
            const uint32_t from = map_to_rank(mine + (uint32_t)((c + h) * kRows * 4), 2 * s + half);
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = ld_cluster1(from + i * kRows * 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] += v[i];
          }
#pragma unroll
          for (int i = 0; i < 8; i += 2) w[(h + i) / 2] = pack16(z[i], z[i + 1], p.fp16);
        }
        store_rows32(p, buf, w, n0, row, lane);
      }
    }
  }

  // (whoever had nothing to wait for: what comes after this kernel comes after the one before it, too)
  depend_wait();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other uses its memory or barriers
  tc_fence_after();
  if (warp == 1) tmem_release<2>(tmem);
}

// ------------------------------------------------------------------ what comes before the products
// Rows put into sorted order, and the maps that end with each group, in one launch.
struct Move {
  const uint4* from;
  uint4* to;
  int rows;           // 0: nothing is moved
  int nvec, pitch;    // 16-byte vectors of a row, and between rows of `to`
  int div, by_slots;  // row p of `to` is row slots[p] / div of `from`, or p
};
struct Setup {
  CUtensorMap d, x;   // maps of dout's and x's sorted rows
  CUtensorMap* ends;  // [2 e] and [2 e + 1]: d and x with their rows cut at the end of group e
  const int32_t *slots, *offsets;
  int E, S;
  int map_blocks, first_blocks;  // blocks (of 8 warps, a warp a map or a row) of the maps, of move[0]
  Move move[2];
};

__device__ __forceinline__ void move_row(const Move& m, const Setup& p, int row, int lane) {
  if (row >= m.rows || row < __ldg(p.offsets) || row >= __ldg(p.offsets + p.E)) return;  // (a row of no group)
  const int slot = m.by_slots ? __ldg(p.slots + row) : row;
  uint4* d = m.to + (size_t)row * m.pitch;
  if (slot < 0 || slot >= p.S) {
    if (lane == 0) record_invalid();
    for (int i = lane; i < m.nvec; i += 32) d[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const uint4* s = m.from + (size_t)(slot / m.div) * m.nvec;
  int i = lane;
  for (; i + 96 < m.nvec; i += 128) {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __ldg(s + i + j * 32);
#pragma unroll
    for (int j = 0; j < 4; ++j) d[i + j * 32] = v[j];
  }
  for (; i < m.nvec; i += 32) d[i] = __ldg(s + i);
}

__global__ void __launch_bounds__(256) grouped_setup_kernel(const __grid_constant__ Setup p) {
  __shared__ __align__(128) CUtensorMap maps[8];
  depend_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int block = blockIdx.x;
  if (block < p.map_blocks) {
    const int i = block * 8 + warp;
    if (i >= 2 * p.E) return;
    const int end = min(max(__ldg(p.offsets + (i >> 1) + 1), 0), p.S);
    CUtensorMap* map = &maps[warp];
    reinterpret_cast<uint32_t*>(map)[lane] = reinterpret_cast<const uint32_t*>(i & 1 ? &p.x : &p.d)[lane];
    __syncwarp();
    if (lane == 0)
      asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(smem_u32(map)), "r"(max(end, 1))
                   : "memory");
    __syncwarp();
    asm volatile(
        "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], [%1], 128;" ::"l"(
            reinterpret_cast<uint64_t>(p.ends + i)),
        "r"(smem_u32(map))
        : "memory");
    return;
  }
  block -= p.map_blocks;
  if (block < p.first_blocks)
    move_row(p.move[0], p, block * 8 + warp, lane);
  else
    move_row(p.move[1], p, (block - p.first_blocks) * 8 + warp, lane);
}

// ------------------------------------------------------------------ host side
// A tensor [outer][rows][inner] in boxes of 128 bytes x box rows of one matrix; outer 0: two dimensions, rows ld apart.
bool make_map(CUtensorMap* m, const void* base, int dtype, long long inner, long long rows, long long outer, int box,
              long long ld = 0) {
  auto enc = get_encode();
  if (!enc) return false;
  const int rank = outer ? 3 : 2, size = dtype == MOE_DT_FP32 ? 4 : 2;
  cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)outer};
  cuuint64_t strides[2] = {(cuuint64_t)(ld ? ld : inner) * size, (cuuint64_t)inner * rows * size};
  cuuint32_t boxes[3] = {(cuuint32_t)(128 / size), (cuuint32_t)box, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType type = dtype == MOE_DT_FP32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : dtype == MOE_DT_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return enc(m, type, rank, const_cast<void*>(base), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Sorted rows: the caller's, or put in order in the workspace, there with a pitch of 128 bytes (rows that start on 128
// bytes are copied at twice the rate of others).
struct Rows {
  const void* at;
  long long ld;
};
long long pitch(long long cols) { return cols > 32 ? (cols + 63) / 64 * 64 : cols; }

// Rows of dout or x [S, cols] as dw takes them, in boxes of 64 rows x 64 columns.  wide: columns in 64s, as [ld / 64][64],
// so that a box takes two neighbouring groups (one behind the other in shared memory) and the two operands of a K block
// are two copies, whose issue bounds the K loop, and not four: 4096 x 14336 over groups of 1024 rows 698 -> 640 us.
// (What lies between cols and ld only reaches sums that are not stored.  dx's weights the same way: no difference.)
bool wide(const Rows& r, long long cols) { return r.ld % 64 == 0 && cols > 128; }
bool make_rows_map(CUtensorMap* m, const Rows& r, int dtype, long long cols, long long S) {
  if (!wide(r, cols)) return make_map(m, r.at, dtype, cols, S, 0, BK, r.ld);
  auto enc = get_encode();
  if (!enc) return false;
  cuuint64_t dims[3] = {64, (cuuint64_t)S, (cuuint64_t)r.ld / 64};
  cuuint64_t strides[2] = {(cuuint64_t)r.ld * 2, 128};
  cuuint32_t boxes[3] = {64, BK, 2};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, dtype == MOE_DT_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
             const_cast<void*>(r.at), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <Mode kMode, bool kPromote, int KS, bool kSplit>
cudaError_t launch(const CUtensorMap& ma, const Maps& mb, const CUtensorMap& mo, const Grouped& g, long long units,
                   int smem, bool overlap, cudaStream_t s) {
  auto kern = grouped_gemm_kernel<kMode, kPromote, KS, kSplit>;
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
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * g.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = overlap_attr();
  cfg.attrs = attr;
  const long long pairs = num_sms() / 2;
  cfg.gridDim = dim3((unsigned)(2 * (g.splits > 1 ? units * g.splits : units < pairs ? units : pairs)));
  cfg.numAttrs = overlap ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, ma, mb, mo, g);
}
template <Mode kMode, bool kPromote>
cudaError_t launch(int ks, const CUtensorMap& ma, const Maps& mb, const CUtensorMap& mo, const Grouped& g,
                   long long units, int smem, bool overlap, cudaStream_t s) {
  if constexpr (kMode != kDw) {
    if (g.splits > 1)
      return ks == 2 ? launch<kMode, kPromote, 2, true>(ma, mb, mo, g, units, smem, overlap, s)
                     : launch<kMode, kPromote, 1, true>(ma, mb, mo, g, units, smem, overlap, s);
    if (ks == 2) return launch<kMode, kPromote, 2, false>(ma, mb, mo, g, units, smem, overlap, s);
  }
  return launch<kMode, kPromote, 1, false>(ma, mb, mo, g, units, smem, overlap, s);
}

// Clusters of `size` CTAs that fit the device at once (a cluster lies within one group of SMs), asked once per device and
// size.
int cluster_slots(int size) {
  static std::atomic<int> cached[64][4];  // (host threads may come at once)
  int dev = 0, log2 = 0;
  while ((1 << log2) < size) ++log2;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = cached[dev][log2].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemMost;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto kern = grouped_gemm_kernel<kForward, false, 1, true>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      n = -1;
    }
    cached[dev][log2].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Columns of a tile at most: narrow ones leave room for more stages where the groups are small, and a group that
// needs a second tile reads its weights twice.  Forward and dx by widths 64 / 128 / 256, us in a graph, groups of random sizes:
// 128 of 1536 x 2048, a mean of 20 rows 126, 122 / 129, 121 / 137, 124; of 28 128, 123 / 131, 122 / 139, 125; of 56 133,
// 126 / 139, 126 / 146, 129; of 72 208, 141 / 144, 129 / 151, 131; of 150 299, 198 / 191, 163 / 171, 142.  16 of 2048 x
// 2048, 24 26.3, 25.8 / 27.5, 25.6 / 29.3, 26.4; 44 27.9, 26.2 / 28.5, 26.1 / 30.3, 27.1; 72 43.6, 31.9 / 30.5, 27.3 /
// 32.0, 28.1.  The cuts lie well below the means where a width loses, because the host does not know the sizes: with
// two thirds of 3000 rows in one of 128 groups 141, 132 / 132, 125 / 135, 128 (64 is taken), of 2000 in one of 64 of
// 4096 x 1024 108, 89 / 95, 84 / 95, 87 (128).  32 or 64 columns for up to 32 rows: within 2 %.
int widest(int S, int E) {
  const int mean = cdiv(S, E);
  return S <= 32 ? 32 : mean <= 24 ? 64 : mean <= 48 ? 128 : 256;
}

// One product.  a: the weights [E, N, K] (dw: not used), b: sorted rows (dw: x's; d: dout's).
template <Mode kMode>
moe_status_t run(const void* a, const Rows& b, const Rows& d, const int32_t* offsets, const int32_t* slots, int to_slots, const int32_t* from,
                 int from_div, int S, int E, int N, int K, int fp16, void* out, int out32, int accumulate, const CUtensorMap* ends, bool overlap, cudaStream_t s) {
  Grouped g = {};
  g.ends = ends;
  g.offsets = offsets;
  g.slots = slots;
  g.to_slots = to_slots;
  g.from = from;
  g.from_div = from_div;
  g.out = out;
  g.S = S;
  g.E = E;
  g.P = kMode == kDx ? K : N;
  g.Q = K;
  g.fp16 = fp16;
  g.out32 = out32;
  g.accumulate = accumulate;
  g.wide_a = kMode == kDw && wide(d, N);
  g.wide_b = kMode == kDw && wide(b, K);
  const int contraction = kMode == kForward ? K : kMode == kDx ? N : S;
  int ks = 1;
  if (kMode == kDw) {
    g.width = K <= 128 ? 128 : 256;
  } else {
    g.width = widest(S, E);
    ks = g.width <= 128 ? 2 : 1;
  }
  while ((1 << g.log2_width) < g.width) ++g.log2_width;
  g.tiles_p = cdiv(g.P, 2 * kRows);
  g.tiles_q = cdiv(g.Q, g.width);
  g.per = g.tiles_p * g.tiles_q;
  g.per_inverse = g.per > 1 ? ~0ull / g.per + 1 : 0;  // (~0 / per is floor(2^64 / per) but for powers of two, where + 1 makes it exact)
  g.KB = cdiv(contraction, BK * ks);
  const int stage = ks * (kRows + g.width / 2) * 128;
  g.stages = (kSmemMost - smem_bytes(kMode, E, 0, 0)) / stage;
  if (g.stages > kMaxStages) g.stages = kMaxStages;
  const int smem = smem_bytes(kMode, E, g.stages, stage);
  const int run = out32 ? kRunFP32 : fp16 ? kRunFP16 : kRunBF16;
  // (the general epilogue of a gradient keeps its sums in fp32 registers)
  const bool promote = cdiv(contraction, BK) > run || out32 || accumulate;
  g.chunk = run / ks;
  g.idesc = make_idesc(fp16 ? 0 : 1, 2 * kRows, 0) | (kMode != kForward ? 1u << 15 : 0) | (kMode == kDw ? 1u << 16 : 0);
  const long long units =
      kMode == kDw ? (long long)E * g.tiles_p * g.tiles_q : (long long)g.tiles_p * (S / g.width + (S < E ? S : E));
  if (units > 1073741823LL) return MOE_ERR_UNSUPPORTED;
  g.splits = 1;
  if (kMode != kDw)
    for (int s = 4; s > 1 && g.splits == 1; s /= 2)
      if (units <= cluster_slots(2 * s) && g.KB - g.KB / s >= kSplitGain) g.splits = s;
  CUtensorMap ma, mo;
  Maps mb;
  const int type = fp16 ? MOE_DT_FP16 : MOE_DT_BF16;
  bool ok;
  if (kMode == kDw) {
    ok = make_map(&mo, out, out32 ? (int)MOE_DT_FP32 : type, K, N, E, 32);
    ma = mo;  // (not used)
  } else {
    ok = make_map(&ma, a, type, K, N, E, kMode == kForward ? kRows : BK * ks);
    if (from) ok = ok && make_map(&mb.b[0], b.at, type, K, S / from_div, 0, 1);
    for (int i = 0; !from && i < g.width / 32; ++i)
      ok = ok && make_map(&mb.b[i], b.at, type, kMode == kForward ? K : N, S, 0, 16 * (i + 1), b.ld);
    mo = ma;  // (not used)
  }
  if (!ok) return MOE_ERR_CUDA;
  const cudaError_t err = promote ? launch<kMode, true>(ks, ma, mb, mo, g, units, smem, overlap, s)
                                  : launch<kMode, false>(ks, ma, mb, mo, g, units, smem, overlap, s);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Where the rows of a tensor in `order` are once they are sorted: at `to` unless they are already.
// Sorted rows that start on no multiple of 128 bytes are worth a copy, too, where there are many and each is read for
// eight tiles or more (cost: two passes over HBM; gain: half of each later copy's time).  As they are / moved, us, forward,
// dx, dw: [1683, 2920] to 13800 in 3 groups 173, 188, 184 / 135, 161, 154; [8192, 2920] to 4096 in 8 212, 164, 163 / 168,
// 164, 150; [2048, 1000] to 2000 in 16 23, 20, 26 / 21, 22, 29; [24824, 5752] to 488 in 32 163 / 207 (forward).
// other: the columns on the products' other side.
bool moved(int order, int S, int cols, int other) {
  return order != MOE_ROWS_SORTED || (pitch(cols) != cols && (long long)S * cols >= 1 << 22 && other >= 2048);
}
Rows placed(const void* from, int order, int S, int cols, int other, void* to) {
  return moved(order, S, cols, other) ? Rows{to, pitch(cols)} : Rows{from, cols};
}
// What puts them there.
Move move_of(const void* from, int order, const Rows& r, int S, int cols, int top_k) {
  return Move{static_cast<const uint4*>(from), static_cast<uint4*>(const_cast<void*>(r.at)), r.at == from ? 0 : S, cols / 8,
              (int)(r.ld / 8), order == MOE_ROWS_TOKEN ? top_k : 1, order != MOE_ROWS_SORTED};
}
// Its launch, if there is anything to do; the next one may then overlap it.
bool set_up(Setup& p, cudaStream_t s) {
  p.map_blocks = p.ends ? cdiv(2 * p.E, 8) : 0;
  p.first_blocks = cdiv(p.move[0].rows, 8);
  const int blocks = p.map_blocks + p.first_blocks + cdiv(p.move[1].rows, 8);
  if (blocks) grouped_setup_kernel<<<blocks, 256, 0, s>>>(p);
  return blocks > 0;
}

size_t rows_bytes(int S, int cols, int other, int order) {
  return !moved(order, S, cols, other) ? 0 : ((size_t)S * pitch(cols) * 2 + 255) / 256 * 256;
}

// The groups' maps, and room to start them on 128 bytes.
size_t maps_bytes(int E) { return (size_t)E * 2 * sizeof(CUtensorMap) + 128; }

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

MOE_DEFINE_STATUS_READER(grouped_wait_status)

moe_status_t grouped_status(int clear) {
  int v = 0;
  const int z = 0;
  if (cudaMemcpyFromSymbol(&v, g_invalid, sizeof(int)) != cudaSuccess) return MOE_ERR_CUDA;
  if (clear && v && cudaMemcpyToSymbol(g_invalid, &z, sizeof(int)) != cudaSuccess) return MOE_ERR_CUDA;
  const moe_status_t waits = grouped_wait_status(clear);
  return waits != MOE_OK ? waits : (moe_status_t)v;
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_grouped_linear_workspace_size(int S, int E, int N, int K, int x_rows) {
  if (S <= 0 || E <= 0 || N <= 0 || K <= 0) return 0;
  return rows_bytes(S, K, N, x_rows);
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
  const size_t need = rows_bytes(S, K, N, x_rows);
  if (need && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // Small groups fetch x's rows by four as they are; putting the rows in order first costs a launch.
  const bool direct = x_rows != MOE_ROWS_SORTED && widest(S, E) <= 64;
  const int div = x_rows == MOE_ROWS_TOKEN ? top_k : 1;
  const Rows xs = direct ? Rows{x, K} : placed(x, x_rows, S, K, N, ws);
  Setup setup = {};
  setup.slots = sorted_slot;
  setup.offsets = expert_offsets;
  setup.E = E;
  setup.S = S;
  setup.move[0] = move_of(x, x_rows, xs, S, K, top_k);
  const bool overlap = set_up(setup, s);
  const bool slots = x_rows != MOE_ROWS_SORTED || out_rows == MOE_ROWS_SLOT;
  const moe_status_t got =
      run<kForward>(w, xs, xs, expert_offsets, slots ? sorted_slot : nullptr, out_rows == MOE_ROWS_SLOT,
                    direct ? sorted_slot : nullptr, div, S, E, N, K, dtype == MOE_DT_FP16, out, 0, 0, nullptr, overlap, s);
  return got == MOE_OK ? launch_status() : got;
}

extern "C" size_t moe_grouped_linear_backward_workspace_size(int S, int E, int N, int K, int dout_rows, int x_rows) {
  if (S <= 0 || E <= 0 || N <= 0 || K <= 0) return 0;
  return rows_bytes(S, N, K, dout_rows) + rows_bytes(S, K, N, x_rows) + maps_bytes(E);
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
  const size_t first = rows_bytes(S, N, K, dout_rows), need = first + (dw ? rows_bytes(S, K, N, x_rows) + maps_bytes(E) : 0);
  if (need && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  const int fp16 = dtype == MOE_DT_FP16;
  uint8_t* next = static_cast<uint8_t*>(ws) + first;  // behind dout's rows
  const Rows d = placed(dout, dout_rows, S, N, K, ws), xs = placed(x, x_rows, S, K, N, next);
  Setup setup = {};
  setup.slots = sorted_slot;
  setup.offsets = expert_offsets;
  setup.E = E;
  setup.S = S;
  setup.move[0] = move_of(dout, dout_rows, d, S, N, top_k);
  if (dw) {
    const int type = fp16 ? MOE_DT_FP16 : MOE_DT_BF16;
    next += rows_bytes(S, K, N, x_rows);
    setup.ends = reinterpret_cast<CUtensorMap*>((reinterpret_cast<uintptr_t>(next) + 127) & ~uintptr_t(127));
    setup.move[1] = move_of(x, x_rows, xs, S, K, top_k);
    if (!make_rows_map(&setup.d, d, type, N, S) || !make_rows_map(&setup.x, xs, type, K, S)) return MOE_ERR_CUDA;
  }
  bool overlap = set_up(setup, s);
  if (dx) {
    const bool slots = dout_rows != MOE_ROWS_SORTED || dx_rows == MOE_ROWS_SLOT;
    st = run<kDx>(w, d, d, expert_offsets, slots ? sorted_slot : nullptr, dx_rows == MOE_ROWS_SLOT, nullptr, 1, S, E, N, K, fp16,
                  dx, 0, 0, nullptr, overlap, s);
    if (st != MOE_OK) return st;
    overlap = true;
  }
  if (dw) {
    st = run<kDw>(nullptr, xs, d, expert_offsets, nullptr, 0, nullptr, 1, S, E, N, K, fp16, dw, out32, accumulate != 0, setup.ends, overlap, s);
    if (st != MOE_OK) return st;
  }
  return launch_status();
}
