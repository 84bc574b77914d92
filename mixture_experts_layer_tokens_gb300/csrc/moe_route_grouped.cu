// moe_route_grouped and its gradient: the router with scores, a balance bias and expert
// groups, one warp per token.
//
//   s_e = sigmoid(l_e) or softmax(l)_e,  c_e = s_e + bias_e,  groups ranked by the sum of
//   their group_top largest c, the top_k largest c of the kept groups chosen,
//   w_j = s_j scale (/ sum of the chosen s).
//
// Lane i holds the NV consecutive experts [i NV, (i + 1) NV) in registers as keys: 32-bit
// integers ordered like the floats, so one redux.sync finds the warp's largest, a ballot the
// lanes that hold it, and the lowest of them holds the lowest index among equals.  A chosen
// key becomes 0, which is below the key of every float.
//
// The order is the one of exact arithmetic.  Without a bias (and, with groups, group_top 1)
// both scores grow with the logit, so the logits themselves are ranked.  With a bias the c
// are computed in fp32, where each is within a known distance of its exact value; if two
// neighbours in the chosen order (the best expert left out and the best group left out among
// them) lie closer than twice that distance and are not equal in logit and bias, the token is
// ranked again in fp64.
#include "moe_vec.cuh"

namespace moe {
namespace {

constexpr int kWarpsPerBlock = 8;
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kMaskedKey = 0x007fffffu;  // the key of -inf: a masked expert

// An unsigned integer ordered like the float (never 0 for a number; -0 counts as +0).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t order_key64(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}

// A logit as the router counts it: NaN as -inf (masked), +inf as the largest finite number.
__device__ __forceinline__ float clean_logit(float x) { return x != x ? -INFINITY : fminf(x, 3.402823466e38f); }

// By exp(-|l|), so that very negative logits keep their relative accuracy.
__device__ __forceinline__ float sigmoid32(float l) {
  const float e = expf(-fabsf(l));
  return __fdiv_rn(l < 0.f ? e : 1.0f, 1.0f + e);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) { return key_value(__reduce_max_sync(kFull, order_key(v))); }

struct RouteArgs {
  const void* logits;
  const float* bias;
  int T, E, top_k;
  int score, n_group, topk_group, group_top, renorm;
  float scale;
};

// The masked state of expert e and its biased score's two inputs.
template <class TL>
__device__ __forceinline__ void expert_inputs(const TL* row, const float* bias, int e, float& l, float& b) {
  l = clean_logit(load1(row + e));
  b = bias ? __ldg(bias + e) : 0.f;
  if (b != b || b == -INFINITY) {
    l = -INFINITY;
    b = 0.f;
  }
}

// ------------------------------------------------------------------ the order in fp64
// Lane j < top_k gets the j-th choice; called by the whole warp.
struct Best64 {
  uint64_t c;
  uint32_t l;
  int i;
};
__device__ __forceinline__ bool better64(const Best64& a, const Best64& b) {
  return a.c != b.c ? a.c > b.c : (a.l != b.l ? a.l > b.l : a.i < b.i);
}
__device__ __forceinline__ Best64 warp_best64(Best64 v) {
#pragma unroll 1
  for (int off = 16; off > 0; off >>= 1) {
    Best64 o;
    o.c = __shfl_xor_sync(kFull, v.c, off);
    o.l = __shfl_xor_sync(kFull, v.l, off);
    o.i = __shfl_xor_sync(kFull, v.i, off);
    if (better64(o, v)) v = o;
  }
  return v;
}

template <int NV, class TL>
__device__ __noinline__ int rank64(const TL* row, const RouteArgs& a) {
  const int lane = threadIdx.x & 31;
  uint64_t c[NV];
  uint32_t lk[NV];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane * NV + i;
    if (e < a.E) m = fmaxf(m, clean_logit(load1(row + e)));
  }
  m = warp_max(m);
  // the softmax's common denominator, in fp64 (sigmoid scores need none)
  double den = 1.0;
  if (a.score == MOE_SCORE_SOFTMAX) {
    den = 0.0;
#pragma unroll 1
    for (int i = 0; i < NV; ++i) {
      const int e = lane * NV + i;
      const float l = e < a.E ? clean_logit(load1(row + e)) : -INFINITY;
      if (l > -INFINITY) den += exp((double)l - (double)m);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) den += __shfl_xor_sync(kFull, den, off);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane * NV + i;
    c[i] = 0;
    lk[i] = 0;
    if (e < a.E) {
      float l, b;
      expert_inputs(row, a.bias, e, l, b);
      lk[i] = order_key(l);
      if (l == -INFINITY) {
        c[i] = order_key64(-INFINITY);
      } else {
        const double s = a.score == MOE_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-(double)l))
                                                      : exp((double)l - (double)m) / den;
        c[i] = order_key64(s + (double)b);
      }
    }
  }
  const uint64_t masked = order_key64(-INFINITY);
  if (a.n_group > 1) {
    const int size = a.E / a.n_group;
    Best64 mine{0, 0, 0x7fffffff};  // lane g: the score of group g
#pragma unroll 1
    for (int g = 0; g < a.n_group; ++g) {
      Best64 first{0, 0, 0x7fffffff}, second;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = lane * NV + i;
        const Best64 v{c[i], 0, e};
        if (e >= g * size && e < (g + 1) * size && better64(v, first)) first = v;
      }
      first = warp_best64(first);
      uint64_t key = first.c;
      if (a.group_top == 2 && first.c != masked) {
        second = Best64{0, 0, 0x7fffffff};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = lane * NV + i;
          const Best64 v{c[i], 0, e};
          if (e >= g * size && e < (g + 1) * size && e != first.i && better64(v, second)) second = v;
        }
        second = warp_best64(second);
        if (second.c != masked) {
          auto val = [](uint64_t k) {
            return __longlong_as_double((long long)(k ^ ((k >> 63) ? 0x8000000000000000ull : ~0ull)));
          };
          key = order_key64(val(first.c) + val(second.c));
        }
      }
      if (lane == g) mine = Best64{key, 0, g};
    }
    uint32_t keep = 0;
#pragma unroll 1
    for (int r = 0; r < a.topk_group; ++r) {
      const Best64 b = warp_best64(mine);
      keep |= 1u << b.i;
      if (lane == b.i) mine = Best64{0, 0, 0x7fffffff};
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane * NV + i;
      if (e < a.E && !((keep >> (e / size)) & 1u)) c[i] = 0;
    }
  }
  int mine = 0;
#pragma unroll 1
  for (int r = 0; r < a.top_k; ++r) {
    Best64 b{0, 0, 0x7fffffff};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Best64 v{c[i], lk[i], lane * NV + i};
      if (c[i] && better64(v, b)) b = v;
    }
    b = warp_best64(b);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane * NV + i == b.i) c[i] = 0;
    if (lane == r) mine = b.i;
  }
  return mine;
}

// ------------------------------------------------------------------ forward
// NV: experts held by a lane (E <= 32 NV).  TL: type of the logits.
template <int NV, class TL>
__global__ void __launch_bounds__(kWarpsPerBlock * 32)
    route_grouped_kernel(const RouteArgs a, int32_t* __restrict__ topk_ids, float* __restrict__ topk_weights) {
  const int t = blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int lane = threadIdx.x & 31;
  const TL* row = static_cast<const TL*>(a.logits) + (size_t)t * a.E;
  const bool by_logit = a.bias == nullptr;

  uint32_t key[NV];
  float l[NV];
  load_lane<NV>(row, a.E, lane, l);
#pragma unroll
  for (int i = 0; i < NV; ++i) l[i] = clean_logit(l[i]);

  // softmax: the row's maximum and denominator (a bias does not enter them; without renormalising the
  // weights need them too)
  float m = 0.f, den = 1.f;
  if (a.score == MOE_SCORE_SOFTMAX && (!by_logit || !a.renorm || a.n_group > 1)) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane * NV + i < a.E) m = fmaxf(m, l[i]);
    m = warp_max(m);
    den = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane * NV + i < a.E && l[i] > -INFINITY) den += expf(l[i] - m);
    den = warp_sum(den);
  }
  auto score32 = [&](float x) {  // s of an unmasked logit
    return a.score == MOE_SCORE_SIGMOID ? sigmoid32(x) : __fdiv_rn(expf(x - m), den);
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane * NV + i;
    key[i] = 0;
    if (e < a.E) {
      if (by_logit) {
        key[i] = order_key(l[i]);
      } else {
        const float b = __ldg(a.bias + e);
        const bool gone = l[i] == -INFINITY || b != b || b == -INFINITY;
        key[i] = gone ? kMaskedKey : order_key(score32(l[i]) + b);
      }
    }
  }
  // Distance below which two fp32 scores may be in the wrong order.  sigmoid: expf is within 1
  // ulp, the sum and the division round once each, so s is within 2^-22 s (s <= 1) and c =
  // s + b within 2^-22 + 2^-24 |c|; two of them, doubled once more for margin.  softmax: the
  // denominator's rounding (up to NV + 5 additions) moves all scores of a row by one common
  // factor within (NV + 6) 2^-24 <= 2^-18.7.
  const float tol0 = a.score == MOE_SCORE_SIGMOID ? 0x1p-20f : 0x1p-17f;
  bool unsure = false;

  if (a.n_group > 1) {
    const int size = a.E / a.n_group;
    uint32_t gkey = 0;  // lane g: the score of group g
#pragma unroll 1
    for (int g = 0; g < a.n_group; ++g) {
      const int e0 = g * size - lane * NV;  // this lane's experts of the group: i in [e0, e0 + size)
      uint32_t k1 = 0, k2 = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t k = (i >= e0 && i < e0 + size) ? key[i] : 0u;
        k2 = max(k2, min(k, k1));
        k1 = max(k1, k);
      }
      const uint32_t top = __reduce_max_sync(kFull, k1);
      uint32_t gk = top;
      if (a.group_top == 2) {
        const uint32_t have = __ballot_sync(kFull, k1 == top);
        const bool owner = lane == __ffs(have) - 1;
        const uint32_t next = __reduce_max_sync(kFull, owner ? k2 : k1);
        if (top != kMaskedKey) {
          float s = key_value(top);
          if (by_logit) s = score32(s);
          if (next > kMaskedKey) s += by_logit ? score32(key_value(next)) : key_value(next);
          gk = order_key(s);
        }
      }
      if (lane == g) gkey = gk;
    }
    uint32_t keep = 0, last = 0, left = 0;
#pragma unroll 1
    for (int r = 0; r < a.topk_group; ++r) {
      last = __reduce_max_sync(kFull, gkey);
      const int w = __ffs(__ballot_sync(kFull, gkey == last)) - 1;
      keep |= 1u << w;
      if (lane == w) gkey = 0;
    }
    left = __reduce_max_sync(kFull, gkey);  // the best group left out (0: none)
    if (!(by_logit && a.group_top == 1) && left != 0 && last != kMaskedKey && left != kMaskedKey) {
      const float x = key_value(last), y = key_value(left);
      unsure |= !(x - y > 2 * tol0 + 0x1p-20f * (fabsf(x) + fabsf(y)));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane * NV + i;
      if (e < a.E && !((keep >> (e / size)) & 1u)) key[i] = 0;
    }
  }

  // top_k rounds, and one more for the best expert left out
  uint32_t my_key = 0;
  int my_id = 0;
  const int rounds = by_logit ? a.top_k : a.top_k + 1;
  uint32_t prev_key = 0;
  int prev_id = 0;
#pragma unroll 1
  for (int r = 0; r < rounds; ++r) {
    uint32_t k1 = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (key[i] > k1) {
        k1 = key[i];
        at = i;
      }
    const uint32_t top = __reduce_max_sync(kFull, k1);
    const int w = __ffs(__ballot_sync(kFull, k1 == top)) - 1;
    const int id = w * NV + __shfl_sync(kFull, at, w);
    if (lane == w)
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i == at) key[i] = 0;
    if (!by_logit && r > 0 && top > kMaskedKey) {
      const float x = key_value(prev_key), y = key_value(top);
      if (!(x - y > tol0 + 0x1p-21f * (fabsf(x) + fabsf(y)))) {
        // equal logit and bias: equal scores, and the lower index came first
        float lx, bx, ly, by;
        expert_inputs(row, a.bias, prev_id, lx, bx);
        expert_inputs(row, a.bias, id, ly, by);
        unsure |= !(lx == ly && bx == by);
      }
    }
    prev_key = top;
    prev_id = id;
    if (lane == r && r < a.top_k) {
      my_key = top;
      my_id = id;
    }
  }
  (void)my_key;
  if (unsure) my_id = rank64<NV, TL>(row, a);

  // weights: lane j has the j-th choice
  float lj = -INFINITY, bj = 0.f;
  if (lane < a.top_k) expert_inputs(row, a.bias, my_id, lj, bj);
  const bool live = lj > -INFINITY;
  float w;
  if (a.renorm) {
    // s_j / sum s is the same for scores scaled by one factor: softmax numerators relative to the
    // largest chosen, sigmoid scores by e^-m (m = the largest chosen logit when all are negative)
    // so that none underflows
    const float top = warp_max(lj);
    float s = 0.f;
    if (live) {
      if (a.score == MOE_SCORE_SOFTMAX)
        s = expf(lj - top);
      else
        s = top < 0.f ? __fdiv_rn(expf(lj - top), 1.0f + expf(lj)) : sigmoid32(lj);
    }
    const float sum = warp_sum(s);
    w = sum > 0.f ? __fdiv_rn(s, sum) : 0.f;
  } else {
    w = live ? score32(lj) : 0.f;
  }
  if (lane < a.top_k) {
    topk_ids[(size_t)t * a.top_k + lane] = my_id;
    topk_weights[(size_t)t * a.top_k + lane] = w * a.scale;
  }
}

// ------------------------------------------------------------------ gradient
// One warp per token; the row is put together in shared memory (zeros, then the chosen
// experts) and written by vectors.
template <int NV, class TL>
__global__ void __launch_bounds__(kWarpsPerBlock * 32)
    route_grouped_backward_kernel(const RouteArgs a, const float* __restrict__ dweights,
                                  const int32_t* __restrict__ topk_ids, TL* __restrict__ dlogits) {
  __shared__ __align__(16) float rows[kWarpsPerBlock][32 * NV];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarpsPerBlock + warp;
  if (t >= a.T) return;
  const TL* row = static_cast<const TL*>(a.logits) + (size_t)t * a.E;
  float* buf = rows[warp];

  int id = -1;
  float dw = 0.f, lj = -INFINITY;
  if (lane < a.top_k) {
    id = topk_ids[(size_t)t * a.top_k + lane];
    dw = dweights[(size_t)t * a.top_k + lane] * a.scale;
    if (id < 0 || id >= a.E) {
      record_status((int)MOE_ERR_INVALID_ARG);
      id = -1;
    } else {
      lj = clean_logit(load1(row + id));
    }
  }
  const bool live = lj > -INFINITY;
  if (!live) dw = 0.f;
  float d = 0.f;
  if (a.renorm) {
    const float top = warp_max(lj);
    float s = 0.f, f = 1.f;
    if (live) {
      if (a.score == MOE_SCORE_SOFTMAX) {
        s = expf(lj - top);
      } else {
        s = top < 0.f ? __fdiv_rn(expf(lj - top), 1.0f + expf(lj)) : sigmoid32(lj);
        f = sigmoid32(-lj);  // 1 - s without the cancellation
      }
    }
    const float sum = warp_sum(s);
    const float p = sum > 0.f ? __fdiv_rn(s, sum) : 0.f;
    const float mean = warp_sum(p * dw);
    d = p * f * (dw - mean);
  } else if (a.score == MOE_SCORE_SIGMOID) {
    if (live) d = dw * sigmoid32(lj) * sigmoid32(-lj);
  }
  float s[NV], dot = 0.f;
  if (!a.renorm && a.score == MOE_SCORE_SOFTMAX) {
    load_lane<NV>(row, a.E, lane, s);
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = clean_logit(s[i]);
      if (lane * NV + i < a.E) m = fmaxf(m, s[i]);
    }
    m = warp_max(m);
    float den = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = (lane * NV + i < a.E && s[i] > -INFINITY) ? expf(s[i] - m) : 0.f;
      den += s[i];
    }
    den = warp_sum(den);
    d = live ? dw * __fdiv_rn(expf(lj - m), den) : 0.f;  // g_j s_j
    dot = warp_sum(d);
    const float rden = den > 0.f ? __fdiv_rn(-dot, den) : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] *= rden;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) buf[lane * NV + i] = s[i];
  __syncwarp();
  // an id chosen twice adds up, in the order of the choices
  const uint32_t same = __match_any_sync(kFull, id < 0 ? -1 - lane : id);
  if (__any_sync(kFull, __popc(same) > 1)) {
    float sum = 0.f;
    for (int j = 0; j < a.top_k; ++j) {
      const float dj = __shfl_sync(kFull, d, j);
      if ((same >> j) & 1u) sum += dj;
    }
    d = sum;
  }
  if (id >= 0 && lane == __ffs(same) - 1) buf[id] += d;
  __syncwarp();
  store_row(dlogits + (size_t)t * a.E, a.E, lane, buf);
}

template <class F>
cudaError_t for_nv(int E, F f) {
  const int nv = (E + 31) / 32;
  if (nv <= 1) return f(std::integral_constant<int, 1>());
  if (nv <= 2) return f(std::integral_constant<int, 2>());
  if (nv <= 4) return f(std::integral_constant<int, 4>());
  if (nv <= 8) return f(std::integral_constant<int, 8>());
  if (nv <= 16) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}

moe_status_t check_route(moe_dtype_t dt, int T, int E, int top_k, const moe_route_config* c) {
  MOE_CHECK_ARG(c && T >= 0 && E >= 1 && E <= 1024 && top_k >= 1 && top_k <= 32);
  MOE_CHECK_ARG(c->n_group >= 1 && c->n_group <= 32 && E % c->n_group == 0);
  MOE_CHECK_ARG(c->topk_group >= 1 && c->topk_group <= c->n_group && top_k <= c->topk_group * (E / c->n_group));
  MOE_CHECK_ARG((c->group_top == 1 || c->group_top == 2) && c->group_top <= E / c->n_group);
  MOE_CHECK_ARG(c->score == MOE_SCORE_SOFTMAX || c->score == MOE_SCORE_SIGMOID);
  MOE_CHECK_ARG(c->scale - c->scale == 0.f);  // finite
  MOE_CHECK_ARG(T <= 2147483647 - kWarpsPerBlock);
  if (dt != MOE_DT_FP32 && dt != MOE_DT_BF16 && dt != MOE_DT_FP16) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

MOE_DEFINE_STATUS_READER(route_grouped_status)

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_route_grouped(const void* logits, moe_dtype_t logits_dtype, const float* bias, int T, int E,
                                          int top_k, const moe_route_config* cfg, int32_t* topk_ids,
                                          float* topk_weights, moe_stream_t stream) {
  const moe_status_t st = check_route(logits_dtype, T, E, top_k, cfg);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  MOE_CHECK_ARG(logits && topk_ids && topk_weights);
  MOE_CHECK_ARG(aligned16(logits) && aligned16(bias) && aligned16(topk_ids) && aligned16(topk_weights));
  const RouteArgs a{logits,          bias,           T,              E,               top_k,     cfg->score,
                    cfg->n_group, cfg->topk_group, cfg->group_top, cfg->renormalize, cfg->scale};
  const dim3 grid((unsigned)((T + kWarpsPerBlock - 1) / kWarpsPerBlock)), block(kWarpsPerBlock * 32);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  for_nv(E, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    if (logits_dtype == MOE_DT_FP32)
      route_grouped_kernel<NV, float><<<grid, block, 0, s>>>(a, topk_ids, topk_weights);
    else if (logits_dtype == MOE_DT_BF16)
      route_grouped_kernel<NV, __nv_bfloat16><<<grid, block, 0, s>>>(a, topk_ids, topk_weights);
    else
      route_grouped_kernel<NV, __half><<<grid, block, 0, s>>>(a, topk_ids, topk_weights);
    return cudaSuccess;
  });
  return launch_status();
}

extern "C" moe_status_t moe_route_grouped_backward(const float* dweights, const void* logits, moe_dtype_t logits_dtype,
                                                   const int32_t* topk_ids, int T, int E, int top_k,
                                                   const moe_route_config* cfg, void* dlogits, moe_stream_t stream) {
  const moe_status_t st = check_route(logits_dtype, T, E, top_k, cfg);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  MOE_CHECK_ARG(dweights && logits && topk_ids && dlogits);
  MOE_CHECK_ARG(aligned16(dweights) && aligned16(logits) && aligned16(topk_ids) && aligned16(dlogits));
  const RouteArgs a{logits,          nullptr,        T,              E,               top_k,     cfg->score,
                    cfg->n_group, cfg->topk_group, cfg->group_top, cfg->renormalize, cfg->scale};
  const dim3 grid((unsigned)((T + kWarpsPerBlock - 1) / kWarpsPerBlock)), block(kWarpsPerBlock * 32);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  for_nv(E, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    if (logits_dtype == MOE_DT_FP32)
      route_grouped_backward_kernel<NV, float>
          <<<grid, block, 0, s>>>(a, dweights, topk_ids, static_cast<float*>(dlogits));
    else if (logits_dtype == MOE_DT_BF16)
      route_grouped_backward_kernel<NV, __nv_bfloat16>
          <<<grid, block, 0, s>>>(a, dweights, topk_ids, static_cast<__nv_bfloat16*>(dlogits));
    else
      route_grouped_backward_kernel<NV, __half>
          <<<grid, block, 0, s>>>(a, dweights, topk_ids, static_cast<__half*>(dlogits));
    return cudaSuccess;
  });
  return launch_status();
}
