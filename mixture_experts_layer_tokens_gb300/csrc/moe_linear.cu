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
// memory, warps 4-11 (two per 32 TMEM lanes) take the other accumulator through the epilogue.
// Problems with fewer tiles than SMs split K over the CTAs of a thread-block cluster: each
// leaves its fp32 partial tile in its own shared memory, and after one cluster barrier every
// CTA adds its share of the elements over distributed shared memory, in rank order.
#include "moe_act.cuh"
#include "moe_mma.cuh"

#include <atomic>

namespace moe {
namespace {

constexpr int BM = 128;           // accumulator rows of a CTA = TMEM lanes
constexpr int BK = 64;            // contraction elements of a K block: one 128-byte swizzle row
constexpr int kThreads = 384;     // three warpgroups: producer and MMA issuer (2 warps idle), 8 epilogue warps
constexpr int kFirstEpi = 4;
constexpr int kEpiWarps = 8;
constexpr int kMaxStages = 16;
constexpr int kStageBudget = 192 * 1024;
constexpr int kCtrlBytes = 512;
constexpr int kSmemBytes = 1024 + kStageBudget + kCtrlBytes + kEpiWarps * 32 * 32 * 4;
// K blocks of a sum in tensor memory, by the output's type: longer ones are promoted (see kPromote)
constexpr int kRunFP32 = 8, kRunFP16 = 128, kRunBF16 = 256;
// kPromote: the epilogue holds up to 128 sums a thread, so the first warpgroup hands it registers
constexpr int kLaunchRegs = 168, kLowRegs = 40, kHighRegs = 232;
static_assert(128 * kLowRegs + 256 * kHighRegs == kThreads * kLaunchRegs, "register split must balance");
static_assert((2 * kMaxStages + 5) * 8 + 4 <= kCtrlBytes && kSmemBytes <= 232448, "shared memory layout");

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
  // the sums rounded to 16 bits and nothing else, by vectors
  __device__ __forceinline__ bool plain() const {
    return !bias && !residual && !preact && act == MOE_LINEAR_NONE && !out32 && Q % 8 == 0;
  }
};

__device__ __forceinline__ void store16(void* p, size_t i, float v, int fp16) {
  if (fp16)
    store1(static_cast<__half*>(p) + i, v);
  else
    store1(static_cast<__nv_bfloat16*>(p) + i, v);
}

// One value, or an aligned pair of adjacent ones, of a 16-bit or fp32 (wide) tensor.
// (plain loads: residual may be out)
__device__ __forceinline__ float load_one(const void* p, size_t at, int fp16, int wide) {
  if (wide) return static_cast<const float*>(p)[at];
  return fp16 ? __half2float(static_cast<const __half*>(p)[at])
              : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
}
__device__ __forceinline__ void store_one(void* p, size_t at, int fp16, int wide, float v) {
  if (wide)
    static_cast<float*>(p)[at] = v;
  else
    store16(p, at, v, fp16);
}
__device__ __forceinline__ void load_pair(const void* p, int fp16, int wide, float (&v)[2]) {
  if (wide) {
    const float2 f = *static_cast<const float2*>(p);
    v[0] = f.x;
    v[1] = f.y;
  } else {
    const uint32_t w = *static_cast<const uint32_t*>(p);
    if (fp16)
      Word<__half>::get(w, v);
    else
      Word<__nv_bfloat16>::get(w, v);
  }
}

// One column of R rows; the loads and stores of the rows are independent.
template <int R>
__device__ __forceinline__ void finish_column(const Epilogue& e, int row, int col, float (&z)[R]) {
  size_t at[R];
  bool valid[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    at[r] = (size_t)(row + r) * e.Q + col;
    valid[r] = row + r < e.P;
  }
  if (e.bias) {
    const float b = load_one(e.bias, col, e.fp16, 0);
#pragma unroll
    for (int r = 0; r < R; ++r) z[r] += b;
  }
  float res[R];
  if (e.residual) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (valid[r]) res[r] = load_one(e.residual, at[r], e.fp16, e.out32);
  }
  if (e.preact) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (valid[r]) store16(e.preact, at[r], z[r], e.fp16);
  }
  if (e.act != MOE_LINEAR_NONE) {
#pragma unroll
    for (int r = 0; r < R; ++r) z[r] = act_fwd(z[r], e.act);
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (valid[r]) store_one(e.out, at[r], e.fp16, e.out32, e.residual ? z[r] + res[r] : z[r]);
}
__device__ __forceinline__ void finish1(const Epilogue& e, int row, int col, float z) {
  float v[1] = {z};
  finish_column(e, row, col, v);
}

// 32 columns x 32 rows of fp32 sums in a warp's shared buffer; 16-byte pieces are placed by
// their index xor the row's low bits, which keeps both the row-per-lane writes and the
// 4-lanes-per-row reads free of bank conflicts.
__device__ __forceinline__ float* buf_at(float* buf, int row, int piece) { return buf + row * 32 + ((piece ^ (row & 7)) << 2); }

template <int act, int R>
__device__ __forceinline__ void act_pairs(float (&z)[R][2]) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    z[r][0] = act_fwd(z[r][0], act);
    z[r][1] = act_fwd(z[r][1], act);
  }
}
// The epilogue of one chunk in the warp's buffer where Q is no multiple of 8, so that a row starts
// anywhere: half a warp takes a row, a lane two columns of every other row that lie in one aligned pair
// of memory.  With an odd Q the pairs of the odd rows (all of the upper half: row0 and col0 are multiples
// of 32) start at odd columns, and 32 elements in all stay single, one a lane.  The loads and stores of 8
// rows are independent, and loaded values are converted after the last load (in the branch of each load
// they cost its latency 8 times: 49 us instead of 32).  [2154, 4070] over 568, the sums alone / with a
// residual / with everything: 26.7 / 31.8 / 44.7 us, by vectors (4072 columns) 18.2 / 23.7 / 33.9.
__device__ __forceinline__ void finish_narrow(const Epilogue& e, float* buf, int row0, int col0, int lane) {
  constexpr int R = 8;
  const int half = lane >> 4, i = lane & 15, n = min(32, e.Q - col0);
  const bool odd = e.Q & 1;
  const int c = 2 * i - (odd && half);  // the lane's columns: c and c + 1
  const bool pair = c >= 0 && c + 1 < n;
  const size_t base = (size_t)(row0 + half) * e.Q + col0 + c;
  auto valid = [&](int h, int r) { return pair && row0 + half + h + 2 * r < e.P; };
  if (odd) {
    // first and last column of the odd rows, or (n odd) the last of the even and the first of the odd ones
    const int row = n & 1 ? lane : 2 * i + 1, col = (n & 1 ? lane & 1 : lane < 16) ? 0 : n - 1;
    finish1(e, row0 + row, col0 + col, buf_at(buf, row, col >> 2)[col & 3]);
  }
  float ba = 0.f, bb = 0.f;
  if (e.bias && pair) {
    ba = load_one(e.bias, col0 + c, e.fp16, 0);
    bb = load_one(e.bias, col0 + c + 1, e.fp16, 0);
  }
  auto put16 = [&](void* p, int h, const float (&z)[R][2]) {
    uint16_t* q = static_cast<uint16_t*>(p) + base;
    uint32_t w[R];
    if (e.fp16) {
#pragma unroll
      for (int r = 0; r < R; ++r) w[r] = Word<__half>::put(z[r]);
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) w[r] = Word<__nv_bfloat16>::put(z[r]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (valid(h, r)) *reinterpret_cast<uint32_t*>(q + (h + 2 * r) * e.Q) = w[r];
  };
#pragma unroll 1
  for (int h = 0; h < 32 && row0 + h < e.P; h += 2 * R) {
    float2 res[R] = {};  // (16-bit types: as loaded, in x; what becomes of it waits for none of the loads)
    if (e.residual) {
      if (e.out32) {
        const float* q = static_cast<const float*>(e.residual) + base;
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (valid(h, r)) res[r] = *reinterpret_cast<const float2*>(q + (h + 2 * r) * e.Q);
      } else {
        const uint16_t* q = static_cast<const uint16_t*>(e.residual) + base;
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (valid(h, r)) res[r].x = *reinterpret_cast<const float*>(q + (h + 2 * r) * e.Q);
      }
    }
    float z[R][2];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = h + 2 * r + half, k = max(c, 0);
      z[r][0] = buf_at(buf, row, k >> 2)[k & 3] + ba;
      z[r][1] = buf_at(buf, row, (c + 1) >> 2)[(c + 1) & 3] + bb;
    }
    if (e.preact) put16(e.preact, h, z);
    if (e.act == MOE_LINEAR_SILU)
      act_pairs<MOE_LINEAR_SILU>(z);
    else if (e.act == MOE_LINEAR_GELU)
      act_pairs<MOE_LINEAR_GELU>(z);
    else if (e.act == MOE_LINEAR_GELU_TANH)
      act_pairs<MOE_LINEAR_GELU_TANH>(z);
    if (e.residual) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float v[2] = {res[r].x, res[r].y};
        if (!e.out32) {
          if (e.fp16)
            Word<__half>::get(__float_as_uint(res[r].x), v);
          else
            Word<__nv_bfloat16>::get(__float_as_uint(res[r].x), v);
        }
        z[r][0] += v[0];
        z[r][1] += v[1];
      }
    }
    if (e.out32) {
      float* q = static_cast<float*>(e.out) + base;
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (valid(h, r)) *reinterpret_cast<float2*>(q + (h + 2 * r) * e.Q) = make_float2(z[r][0], z[r][1]);
    } else {
      put16(e.out, h, z);
    }
  }
}

// 8 consecutive columns (Q % 8 == 0) of R rows, R independent chains of loads and stores;
// `valid` says which rows exist.
template <class T, int R>
__device__ __forceinline__ void add_rows(const void* p, const size_t (&at)[R], const bool (&valid)[R], float (&z)[R][8]) {
  float v[R][8];
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (valid[r]) load8(static_cast<const T*>(p) + at[r], v[r]);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (valid[r]) z[r][i] += v[r][i];
}
template <class T, int R>
__device__ __forceinline__ void store_rows(void* p, const size_t (&at)[R], const bool (&valid)[R], const float (&z)[R][8]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (valid[r]) store8(static_cast<T*>(p) + at[r], z[r]);
}
template <int act, int R>
__device__ __forceinline__ void act_rows(float (&z)[R][8]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 8; ++i) z[r][i] = act_fwd(z[r][i], act);
}
// T: the 16-bit type
template <class T, int R>
__device__ __forceinline__ void finish_rows_as(const Epilogue& e, const int (&row)[R], int col, const bool (&valid)[R],
                                               float (&z)[R][8]) {
  size_t at[R];
#pragma unroll
  for (int r = 0; r < R; ++r) at[r] = (size_t)row[r] * e.Q + col;
  if (e.bias) {
    float b[8];
    load8(static_cast<const T*>(e.bias) + col, b);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 8; ++i) z[r][i] += b[i];
  }
  if (e.preact) store_rows<T>(e.preact, at, valid, z);
  if (e.act == MOE_LINEAR_SILU)
    act_rows<MOE_LINEAR_SILU>(z);
  else if (e.act == MOE_LINEAR_GELU)
    act_rows<MOE_LINEAR_GELU>(z);
  else if (e.act == MOE_LINEAR_GELU_TANH)
    act_rows<MOE_LINEAR_GELU_TANH>(z);
  if (e.out32) {
    if (e.residual) add_rows<float>(e.residual, at, valid, z);
    store_rows<float>(e.out, at, valid, z);
  } else {
    if (e.residual) add_rows<T>(e.residual, at, valid, z);
    store_rows<T>(e.out, at, valid, z);
  }
}
template <int R>
__device__ __forceinline__ void finish_rows(const Epilogue& e, const int (&row)[R], int col, const bool (&valid)[R],
                                            float (&z)[R][8]) {
  if (e.fp16)
    finish_rows_as<__half>(e, row, col, valid, z);
  else
    finish_rows_as<__nv_bfloat16>(e, row, col, valid, z);
}

// ------------------------------------------------------------------ tensor-core kernel
struct Gemm {
  Epilogue e;
  int KB;               // stages of K
  int splits;           // CTAs (CTA pairs) of a cluster that share a tile's K blocks
  int BN;               // tile columns
  int chunk;            // kPromote: stages added up in the tensor memory
  int stages;
  int a_rows;           // rows of the A box (K-major A): with fewer than 128 a stage is smaller and more of
                        // them fit; the MMA reads what lies behind for the other rows, whose
                        // accumulators nobody looks at
  int tiles_m, tiles_n, raster;
  int unit0, units;     // the tiles of this launch: [unit0, units)
  uint32_t idesc;
};

// The tile of a unit: blocks of `raster` tile rows run through all tile columns, so that the CTAs
// that work at the same time share A rows and B rows in L2.
constexpr int kRaster = 8;  // at most; the host evens the blocks out (9 tile rows: 5 and 4, not 8 and a
                            // last row that reads all of B again)
__device__ __forceinline__ void tile_of(const Gemm& p, int u, int& m, int& n) {
  const int per = p.raster * p.tiles_n, g = u / per, in = u - g * per;
  const int rows = min(p.raster, p.tiles_m - g * p.raster);
  m = g * p.raster + in % rows;
  n = in / rows;
}

// The epilogue of one 32-column chunk whose sums lane r holds for row row0 + r.  kPlain: nothing but
// the plain form can come (the gradients).
template <bool kPlain>
__device__ __forceinline__ void finish_chunk(const Epilogue& e, float* buf, const float* v, int row0, int col0, int lane) {
  // 4 lanes to the 32 columns of a row: 64-byte pieces (of 16-bit outputs) of 8 rows at a time
  const int q = lane & 3, col = col0 + q * 8;
  if (kPlain || e.plain()) {
    // rounded before the exchange: half the shared-memory traffic, and short enough that the
    // gate's dx (4 K blocks a tile) went from 38 to 26 us
    char* b16 = reinterpret_cast<char*>(buf);
    auto at = [&](int row, int piece) { return b16 + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4); };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = e.fp16 ? Word<__half>::put(v + 8 * i + 2 * j) : Word<__nv_bfloat16>::put(v + 8 * i + 2 * j);
      *reinterpret_cast<uint4*>(at(lane, i)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
    uint16_t* out = static_cast<uint16_t*>(e.out) + (size_t)row0 * e.Q + col;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + (lane >> 2);
      const uint4 w = *reinterpret_cast<const uint4*>(at(r, q));
      if (row0 + r < e.P && col < e.Q) *reinterpret_cast<uint4*>(out + (size_t)r * e.Q) = w;
    }
    __syncwarp();
    return;
  }
  if constexpr (!kPlain) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<float4*>(buf_at(buf, lane, i)) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    __syncwarp();
    if (e.Q % 8 == 0) {
      if (col < e.Q) {
#pragma unroll
        for (int h = 0; h < 4; h += 2) {  // two rows at a time: four spilled registers
          float z[2][8];
          int row[2];
          bool valid[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = (h + i) * 8 + (lane >> 2);
            const float4 lo = *reinterpret_cast<const float4*>(buf_at(buf, r, q * 2));
            const float4 hi = *reinterpret_cast<const float4*>(buf_at(buf, r, q * 2 + 1));
            z[i][0] = lo.x, z[i][1] = lo.y, z[i][2] = lo.z, z[i][3] = lo.w;
            z[i][4] = hi.x, z[i][5] = hi.y, z[i][6] = hi.z, z[i][7] = hi.w;
            row[i] = row0 + r;
            valid[i] = row[i] < e.P;
          }
          finish_rows<2>(e, row, col, valid, z);
        }
      }
    } else {
      finish_narrow(e, buf, row0, col0, lane);
    }
    __syncwarp();
  }
}

// The share of CTA (pair) `split` of a split tile: its elements summed over the S partial tiles,
// in rank order, through the epilogue.  Called by the epilogue warps.  (Every value that is loaded from
// another CTA is used, so that it has arrived when this one's threads come to the last barrier.)
template <int S, int CG, bool kPlain>
__device__ __forceinline__ void join_splits(const Gemm& p, uint8_t* smem, int unit, int split, int half) {
  int tm, tn;
  tile_of(p, unit, tm, tn);
  const int row0 = (tm * CG + half) * BM;
  const int rows = max(0, min(BM, p.e.P - row0)), cols = min(p.BN, p.e.Q - tn * p.BN);
  const int groups = (cols + 7) / 8, items = rows * groups;
  const uint32_t base = smem_u32(smem);
  const int i1 = (int)((long long)items * (split + 1) / S);
  if (status_failed()) return;
  if (!kPlain && p.e.Q % 8 != 0) {
    // a warp takes 32 columns of four rows at a time
    const int warp = (threadIdx.x >> 5) - kFirstEpi, lane = threadIdx.x & 31, pieces = (cols + 31) / 32;
    const int r0 = rows * split / S, r1 = rows * (split + 1) / S, n = pieces * ((r1 - r0 + 3) / 4);
#pragma unroll 1
    for (int i = warp; i < n; i += kEpiWarps) {
      const int c = i % pieces * 32 + lane, r = r0 + i / pieces * 4;
      float v[4][S] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c < cols && r + j < r1) {
#pragma unroll
          for (int s = 0; s < S; ++s)
            v[j][s] = ld_cluster1(map_to_rank(base + (uint32_t)(((r + j) * (p.BN + 4) + c) * 4), s * CG + half));
        }
      float z[4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int s = 0; s < S; ++s) z[j] += v[j][s];
      // (rows past r1 are another CTA's)
      if (c < cols) {
        if (r + 4 <= r1)
          finish_column(p.e, row0 + r, tn * p.BN + c, z);
        else
          for (int j = 0; j < 4; ++j)
            if (r + j < r1) finish1(p.e, row0 + r + j, tn * p.BN + c, j == 0 ? z[0] : j == 1 ? z[1] : z[2]);
      }
    }
    return;
  }
  constexpr int U = S >= 8 ? 1 : 8 / S;  // items whose loads are in flight together
  constexpr int kStep = kEpiWarps * 32;
  auto some = [&](auto count, int i0) {
    constexpr int C = decltype(count)::value;
    float4 lo[C][S], hi[C][S];
#pragma unroll
    for (int u = 0; u < C; ++u) {
      const int i = i0 + u * kStep, r = i / groups, c = (i - r * groups) * 8;
      const uint32_t at = base + (uint32_t)((r * (p.BN + 4) + c) * 4);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const uint32_t src = map_to_rank(at, s * CG + half);
        lo[u][s] = ld_cluster(src);
        hi[u][s] = ld_cluster(src + 16);
      }
    }
#pragma unroll
    for (int u = 0; u < C; ++u) {
      const int i = i0 + u * kStep, r = i / groups, c = (i - r * groups) * 8;
      float z[1][8] = {};
#pragma unroll
      for (int s = 0; s < S; ++s) {
        z[0][0] += lo[u][s].x, z[0][1] += lo[u][s].y, z[0][2] += lo[u][s].z, z[0][3] += lo[u][s].w;
        z[0][4] += hi[u][s].x, z[0][5] += hi[u][s].y, z[0][6] += hi[u][s].z, z[0][7] += hi[u][s].w;
      }
      const int row[1] = {row0 + r}, col = tn * p.BN + c;
      const bool valid[1] = {true};
      if (kPlain) {
        uint16_t* out = static_cast<uint16_t*>(p.e.out) + (size_t)row[0] * p.e.Q + col;
        if (p.e.fp16)
          store8(reinterpret_cast<__half*>(out), z[0]);
        else
          store8(reinterpret_cast<__nv_bfloat16*>(out), z[0]);
      } else {
        finish_rows<1>(p.e, row, col, valid, z);
      }
    }
  };
  int i = (int)((long long)items * split / S) + threadIdx.x - kFirstEpi * 32;
  if (U > 1)
    for (; i + (U - 1) * kStep < i1; i += U * kStep) some(std::integral_constant<int, U>(), i);
  for (; i < i1; i += kStep) some(std::integral_constant<int, 1>(), i);
}

// kAMN / kBMN: the operand is MN-major (its contraction dimension is the row of its tensor).
// CG: CTAs that share an MMA.  2: a tile has 256 rows, each CTA of the pair copies its 128 rows
//   of A and half of the B rows and holds its rows' accumulators; the even CTA issues the MMAs.
// kPromote: the tensor core adds to its fp32 accumulator by truncation, which over K = 7168 left
//   outputs 8e-6 off (2-norm), and of sums of one sign takes 1.0e-7 a step of 16 elements (measured: 1.0e-4
//   over 16384, 5.9e-3 over a million; fp16 rounds by up to 4.9e-4); so every `chunk` stages the accumulator is
//   added, with rounding, to fp32 sums in the epilogue's registers, and the next block starts from zero in
//   the other accumulator.  fp32 outputs: every 512 elements; fp16 ones every 8192 (5e-5, a tenth of their
//   rounding), bf16 ones every 16384 (1.0e-4, a fortieth), which the K loop nearly hides.
// KS: K blocks of a stage, copied, awaited and multiplied together.  2 where a stage stays at most
//   64 KB: fewer turns of the two loops, which bound narrow tiles ([16, 4096] over K 4096 in
//   64-column tiles 16.5 -> 12.6 us; wider stages lose at 256 columns, 129 -> 150 us for
//   [2050, 8192] over 5120 with one CTA per MMA).
template <bool kAMN, bool kBMN, int CG, bool kPromote, int KS>
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
  float* bufs = reinterpret_cast<float*>(ctrl + kCtrlBytes);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (uniform to the compiler)
  const int stages = p.stages;
  const int bn_cta = p.BN / CG;  // B rows this CTA copies
  const uint32_t a_bytes = kAMN ? 128 * BK * 2 : p.a_rows * 128;
  const uint32_t b_bytes = bn_cta * 128;
  const int a_stage = kAMN ? 128 * 128 : p.a_rows * 128;
  const int stage_bytes = KS * (a_stage + bn_cta * 128);
  const int splits = p.splits;
  const int rank = (CG > 1 || splits > 1) ? (int)cluster_rank() : 0;
  const int half = CG > 1 ? rank & 1 : 0;  // this CTA within its pair
  const int split = rank / CG;
  const uint32_t leader = rank - half;
  const uint16_t pair_mask = (uint16_t)(3u << leader);

  depend_launch();
  if (warp == 2 && elect_one()) {
    prefetch_tensormap(&tmA);
    prefetch_tensormap(&tmB);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kEpiWarps * CG);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_take<CG>(tmem_slot);
  tc_fence_before();
  __syncthreads();
  if (CG > 1) cluster_sync();  // the pair's barriers are set up
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  depend_wait();

  const int kb0 = (int)((long long)p.KB * split / splits), kb1 = (int)((long long)p.KB * (split + 1) / splits);
  const int units = p.units;
  const int first = p.unit0 + blockIdx.x / (splits * CG);
  const int step = splits > 1 ? units : gridDim.x / CG;  // a split tile is its cluster's only work
  const int chunk = kPromote ? p.chunk : kb1 - kb0;  // stages added up in the tensor memory

  if (warp < kFirstEpi) {
    if (kPromote) setmaxnreg_dec<kLowRegs>();
    // The producer's and the MMA issuer's K loops run in one thread chosen by elect.sync, what
    // they need computed outside by the whole warp: with the loop in the warp and its body under
    // `lane == 0` a K block took 640 clocks however narrow the tile (votes each turn, and every
    // operand that copies and MMAs want in uniform registers moved there anew), like this 300.
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
      const uint32_t full0 = CG > 1 ? map_to_rank(smem_u32(full), leader) : smem_u32(full);  // (both CTAs' copies
      for (int u = first; u < units; u += step) {                                           // complete there)
        int tm, tn;
        tile_of(p, u, tm, tn);
        const int arow = (tm * CG + half) * BM, brow = tn * p.BN + half * bn_cta;
        if (elect_one()) {
          int st = stage;
          uint32_t ph = phase;
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!lane_wait(&empty[st], ph ^ 1)) {
              failed = true;
              break;
            }
            uint8_t* sA = smem + st * stage_bytes;
            uint8_t* sB = sA + KS * a_stage;
            const uint32_t bar = full0 + st * 8;
            if (half == 0) mbar_arrive_expect_tx(&full[st], CG * KS * (a_bytes + b_bytes));
            const int k = kb * KS * BK;
            if (kAMN) {
              tma_load<CG>(sA, &tmA, arow, k, bar, pol);
              tma_load<CG>(sA + KS * 8192, &tmA, arow + 64, k, bar, pol);
            } else {
#pragma unroll
              for (int i = 0; i < KS; ++i) tma_load<CG>(sA + i * a_stage, &tmA, k + i * BK, arow, bar, pol);
            }
            if (kBMN) {
              for (int g = 0; g < bn_cta / 64; ++g) tma_load<CG>(sB + g * KS * 8192, &tmB, brow + g * 64, k, bar, pol);
            } else {
#pragma unroll
              for (int i = 0; i < KS; ++i) tma_load<CG>(sB + i * b_bytes, &tmB, k + i * BK, brow, bar, pol);
            }
            if (++st == stages) {
              st = 0;
              ph ^= 1;
            }
          }
          if (failed && half == 0)
            // wait (bounded) for the copies still in flight, of this unit and of the last: each
            // stage's phase that the ring was in
            for (int i = 0; i < stages; ++i)
              mbar_wait(&full[i], i < st ? ph : ph ^ 1, false, 100000000ull);
        }
        __syncwarp();
        if ((failed = __any_sync(0xffffffffu, failed))) break;
        advance(kb1 - kb0);
      }
    } else if (warp == 1 && half == 0) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t a0 = smem_u32(smem), b0 = a0 + KS * a_stage;
      const uint32_t ad0 = desc_lo<kAMN, KS>(a0), bd0 = desc_lo<kBMN, KS>(b0);
      constexpr uint32_t kStepA = (kAMN ? 2048 : 32) >> 4, kStepB = (kBMN ? 2048 : 32) >> 4;  // 16 K elements on
      int acc = 0;
      uint32_t acc_phase = 0;
      for (int u = first; u < units && !failed; u += step) {
        for (int kc = kb0; kc < kb1; kc += chunk) {
          const uint32_t d = tmem + acc * kAccCols;
          const int ke = min(kb1, kc + chunk);
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
                  mma<CG>(d, desc(ad0 + at + i * (kAMN ? 8192 >> 4 : a_stage >> 4) + kk * kStepA),
                          desc(bd0 + at + i * (kBMN ? 8192 >> 4 : b_bytes >> 4) + kk * kStepB), p.idesc,
                          kb > kc || i > 0 || kk > 0);
              commit<CG>(&empty[st], pair_mask);
              if (++st == stages) {
                st = 0;
                ph ^= 1;
              }
            }
            if (!failed) {
              commit<CG>(&tfull[acc], pair_mask);
            } else {
              // a wait gave up: let the MMAs issued so far finish (bounded) before the tensor memory goes
              commit<CG>(drain, pair_mask);
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
    if (splits > 1) cluster_sync();  // (the partial tiles are in shared memory)
    // Every stage comes back before this CTA leaves: the commits of its MMAs arrive on the barriers here, with a
    // pair on those of both CTAs, and the accumulator's barrier, which the epilogue awaited, says nothing about
    // the arrivals of earlier commits.  (It also ends the MMAs that an epilogue which gave up did not await.)
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
    const int side = (warp - kFirstEpi) >> 2;  // column half
    const int ncol = p.BN / 2;
    float* buf = bufs + (warp - kFirstEpi) * 1024;
    const uint32_t tb = tmem + ((uint32_t)(quarter * 32) << 16) + side * ncol;
    const uint32_t freed = CG > 1 ? map_to_rank(smem_u32(tempty), leader) : 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    auto release = [&]() {  // this warp is done with the accumulator
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG > 1)
          mbar_arrive_cluster(freed + acc * 8);
        else
          mbar_arrive(&tempty[acc]);
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    };
    bool ok = true;
    for (int u = first; ok && u < units; u += step) {
      int tm, tn;
      tile_of(p, u, tm, tn);
      const int row0 = (tm * CG + half) * BM + quarter * 32, col0 = tn * p.BN + side * ncol;
      const int cols = row0 < p.e.P ? min(ncol, p.e.Q - col0) : 0;
      // split: the partial tile goes to this CTA's stages (every copy has landed and every MMA has
      // read it when the accumulator is complete)
      float* part = reinterpret_cast<float*>(smem) + (quarter * 32 + lane) * (p.BN + 4) + side * ncol;
      auto take = [&](const float* v, int c) {
        if (splits > 1) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(part + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else {
          finish_chunk<kBMN>(p.e, buf, v, row0, col0 + c, lane);
        }
      };
      if constexpr (kPromote) {
        float sums[128] = {};
        for (int kc = kb0; kc < kb1; kc += chunk) {
          if (!(ok = __all_sync(0xffffffffu, lane_wait(&tfull[acc], acc_phase)))) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 128; c += 32)
            if (c < cols) {
#pragma unroll
              for (int h = 0; h < 32; h += 16) {
                float v[16];
                tmem_ld16(tb + acc * kAccCols + c + h, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) sums[c + h + i] += v[i];
              }
            }
          release();
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 128; c += 32)
          if (c < cols) take(sums + c, c);
      } else {
        if (!(ok = warp_wait(&tfull[acc], acc_phase))) break;
        tc_fence_after();
        for (int c = 0; c < cols; c += 32) {
          float v[32];
          tmem_ld32(tb + acc * kAccCols + c, v);
          tmem_ld_wait();
          take(v, c);
        }
        release();
      }
    }
    if (splits > 1) {
      __syncwarp();
      cluster_sync();  // every CTA's partial tile is in its shared memory
      if (splits == 2)
        join_splits<2, CG, kBMN>(p, smem, first, split, half);
      else if (splits == 4)
        join_splits<4, CG, kBMN>(p, smem, first, split, half);
      else
        join_splits<8, CG, kBMN>(p, smem, first, split, half);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // No CTA leaves while another uses its memory or barriers.  (With splits all that is left to come after
  // the barrier above are the loads of the partial tiles.)
  if (splits > 1)
    cluster_sync_relaxed();
  else if (CG > 1)
    cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_release<CG>(tmem);
}

// ------------------------------------------------------------------ a few rows
// out [kM, N]: each warp takes one weight row (or 1/ks of it) and all rows of x.
// Bound by the weights' bytes; a lane's loads are independent (four vectors of the weights, and of
// each the rows of x: no branch between them, so that they are in flight together), and a CTA has the
// whole of its weight slice on its way.
template <int kM, class T>
__global__ void __launch_bounds__(256)
    linear_rows_kernel(const T* __restrict__ x, const T* __restrict__ w, int N, int K, int ks, const Epilogue e) {
  __shared__ float sums[8][kM];
  constexpr int U = 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = 8 / ks;  // weight rows of the CTA
  const int n = blockIdx.x * per + warp / ks, part = warp % ks;
  float acc[kM] = {};
  if (n < N) {
    const T* wr = w + (size_t)n * K;
    const int step = ks * 256;
    for (int k0 = part * 256; k0 < K; k0 += U * step) {
      float wv[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * step + lane * 8;
        if (k < K) load8(wr + k, wv[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * step + lane * 8;
        if (k < K) {
          float xv[kM][8];
#pragma unroll
          for (int m = 0; m < kM; ++m) load8(x + (size_t)m * K + k, xv[m]);
#pragma unroll
          for (int m = 0; m < kM; ++m)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[m] = fmaf(wv[u][i], xv[m][i], acc[m]);
        }
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
  for (int i = threadIdx.x; i < per * kM; i += blockDim.x) {
    const int r = i % per, m = i / per, col = blockIdx.x * per + r;
    if (col >= N) continue;
    float z = 0.f;
    for (int s = 0; s < ks; ++s) z += sums[r * ks + s][m];
    finish1(e, m, col, z);
  }
}

// ------------------------------------------------------------------ dz and its column sums
// dz = dout * act'(preact), in the operand type (row stride ld), and one row of column sums per
// chunk of rows.  A thread takes V columns (8, or 2 or 1 where N is no multiple of 8) of every 8th row of its
// chunk.
constexpr int kDzRows = 64;       // rows of a chunk, fewer where that leaves SMs idle, more where it
constexpr int kDzChunks = 1024;   // would give over this many chunks

template <int V, class T>
__device__ __forceinline__ void load_cols(const T* p, float (&v)[V]) {
  if constexpr (V == 8)
    load8(p, v);
  else if constexpr (V == 2)
    load_pair(p, std::is_same<T, __half>::value, std::is_same<T, float>::value, v);
  else
    v[0] = load1(p);
}

template <class TO, class T, int V, int act>
__global__ void __launch_bounds__(256, 4)
    linear_dz_kernel(const TO* __restrict__ dout, const T* __restrict__ preact, int M, int N, T* __restrict__ dz,
                     int ld, int rows, float* __restrict__ partial) {
  constexpr int R = V == 2 ? 4 : 2;  // rows whose loads are in flight together
  depend_launch();
  __shared__ float sums[8][32 * V];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int col = (blockIdx.x * 32 + cx) * V;
  const int r0 = blockIdx.y * rows, r1 = min(M, r0 + rows);
  float sum[V] = {};
  if (col < N)
    for (int rb = r0 + ry; rb < r1; rb += 8 * R) {
      float d[R][V], z[R][V];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int r = rb + 8 * j;
        if (r >= r1) break;
        const size_t at = (size_t)r * N + col;
        load_cols(dout + at, d[j]);
        if (act != MOE_LINEAR_NONE) load_cols(preact + at, z[j]);
      }
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int r = rb + 8 * j;
        if (r >= r1) break;
        if (act != MOE_LINEAR_NONE) {
#pragma unroll
          for (int i = 0; i < V; ++i) d[j][i] *= act_grad(z[j][i], act);
        }
        if (dz) {
          T* p = dz + (size_t)r * ld + col;
          if constexpr (V == 8)
            store8(p, d[j]);
          else if constexpr (V == 2)
            *reinterpret_cast<uint32_t*>(p) = Word<T>::put(d[j]);
          else
            store1(p, d[j][0]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] += d[j][i];
      }
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
  depend_launch();
  depend_wait();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  float s = 0.f;
  if (c < N)
#pragma unroll 8
    for (int p = part; p < P; p += 8) s += partial[(size_t)p * N + c];
  sums[part][threadIdx.x & 31] = s;
  __syncthreads();
  if (part == 0 && c < N) {
    for (int i = 1; i < 8; ++i) s += sums[i][threadIdx.x & 31];
    store1(dbias + c, s);
  }
}

// ------------------------------------------------------------------ host side
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

template <bool kAMN, bool kBMN, int CG, bool kPromote, int KS>
cudaError_t launch_gemm(const CUtensorMap& ma, const CUtensorMap& mb, const Gemm& g, int grid, bool overlap, cudaStream_t s) {
  auto kern = linear_gemm_kernel<kAMN, kBMN, CG, kPromote, KS>;
  if (kPromote) {
    // The epilogue's warps take more registers than a thread is launched with (setmaxnreg), from those that the
    // first warpgroup gives back: a build with fewer than kLaunchRegs would wait for them without an end, so
    // it never launches.
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
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = g.splits * CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = overlap_attr();
  cfg.attrs = attr;
  cfg.numAttrs = overlap ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, ma, mb, g);
}

template <bool kAMN, bool kBMN, bool kPromote>
cudaError_t launch_gemm(int cg, int ks, const CUtensorMap& ma, const CUtensorMap& mb, const Gemm& g, int grid,
                        bool overlap, cudaStream_t s) {
  if (cg == 2)
    return ks == 2 ? launch_gemm<kAMN, kBMN, 2, kPromote, 2>(ma, mb, g, grid, overlap, s)
                   : launch_gemm<kAMN, kBMN, 2, kPromote, 1>(ma, mb, g, grid, overlap, s);
  return ks == 2 ? launch_gemm<kAMN, kBMN, 1, kPromote, 2>(ma, mb, g, grid, overlap, s)
                 : launch_gemm<kAMN, kBMN, 1, kPromote, 1>(ma, mb, g, grid, overlap, s);
}

template <bool kAMN, bool kBMN>
cudaError_t launch_gemm(bool promote, int cg, int ks, const CUtensorMap& ma, const CUtensorMap& mb, const Gemm& g,
                        int grid, bool overlap, cudaStream_t s) {
  return promote ? launch_gemm<kAMN, kBMN, true>(cg, ks, ma, mb, g, grid, overlap, s)
                 : launch_gemm<kAMN, kBMN, false>(cg, ks, ma, mb, g, grid, overlap, s);
}

// Clusters of `size` GEMM CTAs that fit the device at once (a cluster lies within one group of
// SMs, so eight-CTA clusters leave SMs idle); asked once per device and size.
int cluster_slots(int size) {
  static std::atomic<int> cached[64][4];  // (host threads may come at once)
  int dev = 0, log2 = 0;
  while ((1 << log2) < size) ++log2;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return num_sms() / size;
  int n = cached[dev][log2].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto kern = linear_gemm_kernel<false, false, 1, false, 1>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      n = num_sms() / size;
    }
    cached[dev][log2].store(n, std::memory_order_relaxed);
  }
  return n;
}

// How a product is cut: CTAs per MMA, tile columns, CTAs (pairs) that share a tile's K.
struct Plan {
  int cg, bn, splits;
};

// The cheapest cut by a model fitted to measurements (ns, at 1.9 GHz): a K block takes 140 (the MMAs
// read 128 rows of A from shared memory whatever the columns) or 1.06 a column (the MMA rate) or 8 a KB
// copied (the SM's port to L2; 16 where the operand's rows do not start on 128 bytes: every row of a
// box then lies in two lines), 15 % less when fewer SMs copy; a tile's epilogue 1200 (1800 with pairs)
// + 12 a column, overlapped with the next tile's K loop; joining split tiles 1500 and its bytes at 10 a
// ns.  Measured either side of it: [64, 256] over K 7168 in 64-column tiles, 1 / 2 / 4 / 8 splits 26 /
// 16 / 11 / 8.9 us; [4096, 256] over 7168 to fp32, (one CTA an MMA, 128 columns, 2 splits) 23.3, (one,
// 256, 4) 25.2, (pairs, 128, 2) 21.5; [8192, 4096] over 4096, one CTA or a pair per MMA 174 / 152;
// [512, 4096] over 4096 in 128 columns, one CTA / a pair 20.5 / 18.0; and by the rows' pitch:
// [2154, 4064] over 568, (one, 128) / (one, 256) / (pairs, 256) 27.9 / 20.7 / 18.0, over 576 13.
Plan plan_gemm(long long P, long long Q, int KB, double a_kb, double b_kb) {
  Plan best{1, 64, 1};
  double best_cost = 1e30;
  const double rows = P < BM ? (double)P : (double)BM;
  for (int cg = 1; cg <= 2; ++cg)
    for (int bn = 64; bn <= 256; bn *= 2) {
      if (cg == 2 && (P <= 128 || bn < 128)) continue;
      const long long tiles = (long long)cdiv(P, BM * cg) * cdiv(Q, bn);
      for (int s = 1; s * cg <= 8; s *= 2) {
        const int slots = cluster_slots(s * cg);
        if (s > 1 && (KB < 4 * s || tiles > slots)) break;
        const double busy = (double)(tiles < slots ? tiles : slots) * s * cg / num_sms();
        const double copy = (rows * a_kb + bn / cg * b_kb) * 0.125 * (busy > 0.85 ? busy : 0.85);
        double kb = 1.06 * bn > copy ? 1.06 * bn : copy;
        if (kb < 140) kb = 140;
        const double loop = cdiv(KB, s) * kb, epi = 600 * (1 + cg) + 12.0 * bn;
        const double waves = cdiv(tiles, slots);
        const double join = s > 1 ? 1500 + rows * bn * 4 * (s - 1) / s / 10 : 0;
        const double cost = waves * (loop > epi ? loop : epi) + (loop > epi ? epi : loop) + join;
        if (cost < best_cost) {
          best_cost = cost;
          best = {cg, bn, s};
        }
      }
    }
  return best;
}

// Splits of the last, partly filled wave of tiles: `rem` tiles that would leave the other slots idle
// for a whole K loop take a launch of their own, several CTAs (pairs) to a tile, when at the MMA rate
// that saves 8 us: its launch and join cost about 6 of them.  (The dense dx of
// 2050 x 5120 over 8192, 152 tiles and 28 more on 76 pairs, 122 -> 117 us.)
int tail_splits(const Plan& p, long long rem, int KB) {
  int s = 1;
  while (2 * s * p.cg <= 8 && rem <= cluster_slots(2 * s * p.cg) && KB >= 16 * s) s *= 2;
  return (double)KB * (1.0 - 1.0 / s) * 1.06 * p.bn > 8000 ? s : 1;
}

// D [P, Q] = A . B^T over a contraction of C.  overlap: what ran before on the stream in this call
// is this library's, so the launch may overlap its end (the kernel waits for its results).
moe_status_t run_gemm(const Operand& A, const Operand& B, int C, const Epilogue& e, bool overlap, cudaStream_t s) {
  Gemm g;
  g.e = e;
  g.KB = cdiv(C, BK);
  auto kb_ns = [](const Operand& o) { return o.ld % 64 || reinterpret_cast<uintptr_t>(o.base) % 128 ? 16.0 : 8.0; };
  const Plan p = plan_gemm(e.P, e.Q, g.KB, kb_ns(A), kb_ns(B));
  g.tiles_m = cdiv(e.P, BM * p.cg);
  g.tiles_n = cdiv(e.Q, p.bn);
  g.raster = cdiv(g.tiles_m, cdiv(g.tiles_m, kRaster));
  g.BN = p.bn;
  const long long units = (long long)g.tiles_m * g.tiles_n;
  if (units > 2147483647LL / 16) return MOE_ERR_UNSUPPORTED;
  g.a_rows = A.mn || e.P >= BM ? BM : (e.P + 7) / 8 * 8;
  const int ks = p.bn <= 128 ? 2 : 1;
  const int blocks = g.KB;
  g.KB = cdiv(blocks, ks);
  g.stages = kStageBudget / (ks * (g.a_rows + p.bn / p.cg) * 128);
  if (g.stages > kMaxStages) g.stages = kMaxStages;
  // a tile of the launch that does not split K, or splits it least, has the longest sums
  const int run = e.out32 ? kRunFP32 : e.fp16 ? kRunFP16 : kRunBF16;
  const bool promote = e.out32 ? blocks > run : cdiv(blocks, p.splits) > run;
  g.chunk = run / ks;
  g.idesc = make_idesc(e.fp16 ? 0 : 1, BM * p.cg, p.bn) | (A.mn ? 1u << 15 : 0) | (B.mn ? 1u << 16 : 0);
  CUtensorMap ma, mb;
  const bool ok = (A.mn ? make_map(&ma, A.base, e.fp16, e.P, C, A.ld, BK * ks)
                        : make_map(&ma, A.base, e.fp16, C, e.P, A.ld, g.a_rows)) &&
                  (B.mn ? make_map(&mb, B.base, e.fp16, e.Q, C, B.ld, BK * ks)
                        : make_map(&mb, B.base, e.fp16, C, e.Q, B.ld, p.bn / p.cg));
  if (!ok) return MOE_ERR_CUDA;
  auto launch = [&](long long first, long long last, int splits) {
    g.unit0 = (int)first;
    g.units = (int)last;
    g.splits = splits;
    const long long ctas = (last - first) * splits * p.cg;
    const int most = cluster_slots(p.cg) * p.cg;
    const int grid = (int)(splits > 1 || ctas < most ? ctas : most);
    const cudaError_t err = A.mn   ? launch_gemm<true, true>(promote, p.cg, ks, ma, mb, g, grid, overlap, s)
                            : B.mn ? launch_gemm<false, true>(promote, p.cg, ks, ma, mb, g, grid, overlap, s)
                                   : launch_gemm<false, false>(promote, p.cg, ks, ma, mb, g, grid, overlap, s);
    overlap = true;
    return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  };
  const int slots = cluster_slots(p.cg);
  const long long rem = p.splits == 1 && units > slots ? units % slots : 0;
  const int tail = rem ? tail_splits(p, rem, blocks) : 1;
  if (tail == 1) return launch(0, units, p.splits);
  const moe_status_t st = launch(0, units - rem, 1);
  return st != MOE_OK ? st : launch(units - rem, units, tail);
}

template <int kM>
void launch_rows(const void* x, const void* w, int N, int K, const Epilogue& e, cudaStream_t s) {
  int ks = 1;
  while (ks < 8 && (long long)N * ks < 16LL * num_sms() && ks * 512 <= K) ks *= 2;
  const int grid = cdiv(N, 8 / ks);
  if (e.fp16)
    linear_rows_kernel<kM, __half>
        <<<grid, 256, 0, s>>>(static_cast<const __half*>(x), static_cast<const __half*>(w), N, K, ks, e);
  else
    linear_rows_kernel<kM, __nv_bfloat16>
        <<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(w), N, K, ks, e);
}

struct BwdLayout {
  long long ld;
  int rows, chunks;  // of linear_dz_kernel
  size_t partial, total;
};
int dz_cols(int N) { return N % 8 == 0 ? 8 : N % 2 == 0 ? 2 : 1; }  // columns a thread of linear_dz_kernel
BwdLayout bwd_layout(int M, int N) {
  BwdLayout l;
  // Rows of dz on 128 bytes copy at more than twice the rate of others (TMA wants 16), but narrow ones grow the
  // workspace by a factor for little: [4096, N] to 7168 in a graph, us at 16 / 128 bytes: N 16 36.8 / 36.1,
  // 24 41.2 / 39.0, 56 47.8 / 38.8, 72 53.9 / 47.7, 200 54.2 / 47.8; [16384, 8] to 2048 75.7 / 81.5.
  const int pitch = N > 32 ? 64 : 8;
  l.ld = ((long long)N + pitch - 1) / pitch * pitch;
  l.rows = kDzRows;
  const int blocks = cdiv(N, 32 * dz_cols(N));
  while (l.rows > 8 && (long long)blocks * cdiv(M, l.rows) < 4LL * num_sms()) l.rows /= 2;
  while (cdiv(M, l.rows) > kDzChunks) l.rows *= 2;
  l.chunks = cdiv(M, l.rows);
  l.partial = ((size_t)M * l.ld * 2 + 255) / 256 * 256;
  l.total = l.partial + (size_t)l.chunks * N * sizeof(float);
  return l;
}

template <class TO, class T, int act>
void launch_dz_act(const TO* d, const T* z, int M, int N, T* dz, const BwdLayout& l, float* partial, cudaStream_t s) {
  auto go = [&](auto v) {
    constexpr int V = decltype(v)::value;
    linear_dz_kernel<TO, T, V, act>
        <<<dim3(cdiv(N, 32 * V), l.chunks), 256, 0, s>>>(d, z, M, N, dz, (int)l.ld, l.rows, partial);
  };
  const int cols = dz_cols(N);
  if (cols == 8)
    go(std::integral_constant<int, 8>());
  else if (cols == 2)
    go(std::integral_constant<int, 2>());
  else
    go(std::integral_constant<int, 1>());
}
template <class TO, class T>
void launch_dz(const void* dout, const void* preact, int M, int N, int act, void* dz, const BwdLayout& l, float* partial,
               cudaStream_t s) {
  const TO* d = static_cast<const TO*>(dout);
  const T* z = static_cast<const T*>(preact);
  T* o = static_cast<T*>(dz);
  switch (act) {
    case MOE_LINEAR_NONE: return launch_dz_act<TO, T, MOE_LINEAR_NONE>(d, z, M, N, o, l, partial, s);
    case MOE_LINEAR_SILU: return launch_dz_act<TO, T, MOE_LINEAR_SILU>(d, z, M, N, o, l, partial, s);
    case MOE_LINEAR_GELU: return launch_dz_act<TO, T, MOE_LINEAR_GELU>(d, z, M, N, o, l, partial, s);
    default: return launch_dz_act<TO, T, MOE_LINEAR_GELU_TANH>(d, z, M, N, o, l, partial, s);
  }
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
  // Few rows: dot products start 3 us sooner than the tensor cores, which win once there is work.  In a
  // graph, rows / GEMM in us: [4, 256] over 7168 4.4 / 7.9, [8, 256] 6.7 / 8.0, [8, 256] over 12288 9.1 /
  // 9.9; [4, 1024] over 4096 7.2 / 6.9, [5, 4096] over 1024 7.6 / 7.8, [3, 1024] over 7168 8.6 / 8.4;
  // [1, 4096] over 4096 6.4 / 9.0, [2, 4096] 8.8 / 9.1, [1, 14336] 30.4 / 24.7.
  if (M <= 8 && (long long)M * N * K <= (M <= 2 ? 34000000 : 20000000)) {
    switch (M) {
      case 1: launch_rows<1>(x, w, N, K, e, s); break;
      case 2: launch_rows<2>(x, w, N, K, e, s); break;
      case 3: launch_rows<3>(x, w, N, K, e, s); break;
      case 4: launch_rows<4>(x, w, N, K, e, s); break;
      case 5: launch_rows<5>(x, w, N, K, e, s); break;
      case 6: launch_rows<6>(x, w, N, K, e, s); break;
      case 7: launch_rows<7>(x, w, N, K, e, s); break;
      default: launch_rows<8>(x, w, N, K, e, s); break;
    }
    return launch_status();
  }
  return run_gemm({x, false, K}, {w, false, K}, K, e, false, s);
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
      const cudaError_t err =
          fp16 ? launch_overlapped(linear_dbias_kernel<__half>, cdiv(N, 32), 256, s, (const float*)partial, l.chunks, N,
                                   static_cast<__half*>(dbias))
               : launch_overlapped(linear_dbias_kernel<__nv_bfloat16>, cdiv(N, 32), 256, s, (const float*)partial,
                                   l.chunks, N, static_cast<__nv_bfloat16*>(dbias));
      if (err != cudaSuccess) return MOE_ERR_CUDA;
    }
    if ((st = launch_status()) != MOE_OK) return st;
  }
  const void* z = direct ? dout : dz;
  const long long ld = direct ? N : l.ld;
  if (dx) {
    const Epilogue e{nullptr, nullptr, dx, nullptr, M, K, MOE_LINEAR_NONE, fp16, 0};
    if ((st = run_gemm({z, false, ld}, {w, true, K}, N, e, dz || partial, s)) != MOE_OK) return st;
  }
  if (dw) {
    const Epilogue e{nullptr, nullptr, dw, nullptr, N, K, MOE_LINEAR_NONE, fp16, 0};
    if ((st = run_gemm({z, true, ld}, {x, true, K}, M, e, dz || partial || dx, s)) != MOE_OK) return st;
  }
  return launch_status();
}
