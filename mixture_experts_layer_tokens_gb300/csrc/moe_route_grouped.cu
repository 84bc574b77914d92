// moe_route_grouped and its gradient: the router with scores, a balance bias and expert
// groups, one warp per token.
//
//   s_e = sigmoid(l_e) or softmax(l)_e,  c_e = s_e + bias_e,  groups ranked by the sum of
//   their group_top largest c, the top_k largest c of the kept groups chosen,
//   w_j = s_j scale (/ sum of the chosen s).
//
// Layout: the 32 lanes are dealt to the groups, a power of two of them to each, and a lane
// holds up to NV consecutive experts of its group, so a group's sums need a few shuffles among
// its own lanes and a lower lane always holds lower experts.  A lane keeps its experts as
// 32-bit keys ordered like the floats, the low bits replaced by the place within the lane, and
// sorts them once; a round of the choice is then one redux.sync over the lanes' first keys, a
// ballot, and a shift of the winner's list.
//
// The order is the one of fp64 arithmetic.  Without a bias both scores grow with the logit, so
// the logits themselves are ranked.  With a bias the c are computed in fp32, where each is
// within a known distance of its exact value (the replaced bits included); if two neighbours in
// the chosen order (the best expert left out and the best group left out among them) lie closer
// than that and are not equal in logit and bias, those that could be chosen, one a lane, are
// ranked from scores held as pairs of floats (2^-39); what that does not settle is ranked from
// scratch in pairs and at last in fp64.  fp64 at once cost about 20 us for such a token (the
// tensor of 16384 tokens has some 20 of them in doubt): this machine does two fp64 FMAs a clock
// per SM.
#include "moe_vec.cuh"

namespace moe {
namespace {

constexpr int kWarpsPerBlock = 8;
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kMaskedKey = 0x007fffffu;  // the key of -inf: a masked expert

// An unsigned integer ordered like the float (never 0 for a number; -0 counts as +0).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// A logit as the router counts it: NaN as -inf (masked), +inf as the largest finite number.
__device__ __forceinline__ float clean_logit(float x) {
  return fminf(fmaxf(x, -INFINITY), 3.402823466e38f);  // (the maximum of a NaN and a number is the number)
}

// By exp(-|l|), so that very negative logits keep their relative accuracy.
__device__ __forceinline__ float sigmoid32(float l) {
  const float e = expf(-fabsf(l));
  return __fdividef(l < 0.f ? e : 1.0f, 1.0f + e);  // (the divisor lies in [1, 2])
}

// exp(l - m) for l <= m, the rounding of the difference made good (it is |l - m| 2^-24 of the result).
__device__ __forceinline__ float exp_below(float l, float m) {
  const float d = l - m;
  if (!(d > -200.f)) return 0.f;
  const float t = __fsub_rn(d, l);  // the error of d by Knuth's two-sum
  const float err = __fsub_rn(__fsub_rn(l, __fsub_rn(d, t)), __fadd_rn(m, t));
  const float e = expf(d);
  return fmaf(e, err, e);
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
  int size;  // experts of a group
  int lpg;   // lanes of a group: the largest power of two that gives every group as many
};

// Logit and bias of expert e, the masked state folded into the logit.
template <class TL>
__device__ __forceinline__ void expert_inputs(const TL* row, const float* bias, int e, float& l, float& b) {
  l = clean_logit(load1(row + e));
  b = bias ? __ldg(bias + e) : 0.f;
  if (b != b || b == -INFINITY) l = -INFINITY;
  if (l == -INFINITY) b = 0.f;  // (masked experts are all alike)
}

// ------------------------------------------------------------------ pairs of floats
// hi + lo with |lo| at most half a last place of hi; the error terms of sums and products by
// the classical two-sum (Knuth) and by fma.
struct FF {
  float h, l;
};
__device__ __forceinline__ FF two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ FF norm(float h, float l) {
  const float s = __fadd_rn(h, l);
  return {s, __fsub_rn(l, __fsub_rn(s, h))};
}
__device__ __forceinline__ FF add(FF a, FF b) {
  const FF s = two_sum(a.h, b.h);
  return norm(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ FF mul(FF a, FF b) {
  const float p = __fmul_rn(a.h, b.h);
  return norm(p, __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, __fmaf_rn(a.h, b.h, -p))));
}
__device__ __forceinline__ FF div(FF a, FF b) {
  const float q = __fdiv_rn(a.h, b.h);
  const FF r = add(a, mul({-q, 0.f}, b));
  return norm(q, __fdiv_rn(r.h, b.h));
}
// exp of a pair <= 0 to about 2^-45: n ln 2 taken off (ln 2 as 12 + 12 + 24 bits, so that its
// products with n are exact), Taylor's series for the rest, |r| <= 0.35: the terms from r^8 / 8!
// in fp32, below them in pairs.
__device__ __noinline__ FF exp_ff(FF a) {
  if (!(a.h > -150.f)) return {0.f, 0.f};  // below every fp32 number
  const float n = rintf(a.h * 1.4426950408889634f);
  FF r = two_sum(__fmaf_rn(-n, 0.693115234375f, a.h), -n * 3.1948089599609375e-05f);
  r = norm(r.h, __fadd_rn(r.l, __fmaf_rn(-n, -1.9046542e-09f, a.l)));
  float q = 1.60590444e-10f;
  q = __fmaf_rn(q, r.h, 2.08767559e-09f);
  q = __fmaf_rn(q, r.h, 2.50521079e-08f);
  q = __fmaf_rn(q, r.h, 2.755732e-07f);
  q = __fmaf_rn(q, r.h, 2.75573188e-06f);
  q = __fmaf_rn(q, r.h, 2.48015876e-05f);
  FF s = add({0.000198412701f, -2.72559687e-12f}, mul(r, {q, 0.f}));
  s = add({0.00138888892f, -3.36310944e-11f}, mul(r, s));
  s = add({0.00833333377f, -4.34617203e-10f}, mul(r, s));
  s = add({0.0416666679f, -1.24176347e-09f}, mul(r, s));
  s = add({0.166666672f, -4.96705388e-09f}, mul(r, s));
  s = add({0.5f, 0.f}, mul(r, s));
  s = add({1.f, 0.f}, mul(r, s));
  s = add({1.f, 0.f}, mul(r, s));
  return {ldexpf(s.h, (int)n), ldexpf(s.l, (int)n)};
}

// ------------------------------------------------------------------ the order from exact scores
// The two precisions of the second ranking: a value type, the score, and keys ordered like it.
struct PairScores {
  using V = FF;
  static __device__ __forceinline__ V of(float x) { return {x, 0.f}; }
  static __device__ __forceinline__ V plus(V a, V b) { return add(a, b); }
  static __device__ V exp_diff(float l, float m) { return exp_ff(two_sum(l, -m)); }
  static __device__ V quotient(V a, V b) { return div(a, b); }
  static __device__ __forceinline__ V shfl(V v, int off) {
    return {__shfl_xor_sync(kFull, v.h, off), __shfl_xor_sync(kFull, v.l, off)};
  }
  static __device__ __forceinline__ uint64_t key(V v) { return ((uint64_t)order_key(v.h) << 32) | order_key(v.l); }
  static __device__ __forceinline__ V value(uint64_t k) { return {key_value((uint32_t)(k >> 32)), key_value((uint32_t)k)}; }
  // x >= y cannot be told from y (the scores are within 2^-42 or so of the exact ones)
  static __device__ bool near(uint64_t kx, uint64_t ky, float more = 0.f) {
    const FF x = value(kx), y = value(ky);
    return !((x.h - y.h) + (x.l - y.l) > more + 0x1p-39f + 0x1p-40f * (fabsf(x.h) + fabsf(y.h)));
  }
};
struct DoubleScores {
  using V = double;
  static __device__ __forceinline__ V of(float x) { return x; }
  static __device__ __forceinline__ V plus(V a, V b) { return a + b; }
  static __device__ V exp_diff(float l, float m) { return exp((double)l - (double)m); }
  static __device__ V quotient(V a, V b) { return a / b; }
  static __device__ __forceinline__ V shfl(V v, int off) { return __shfl_xor_sync(kFull, v, off); }
  static __device__ __forceinline__ uint64_t key(V v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
  }
  static __device__ __forceinline__ V value(uint64_t k) {
    return __longlong_as_double((long long)(k ^ ((k >> 63) ? 0x8000000000000000ull : ~0ull)));
  }
  static __device__ bool near(uint64_t, uint64_t, float = 0.f) { return false; }  // equal ones go by logit and index
};

constexpr uint64_t kMasked64 = 1;  // below the key of every number, above a chosen expert's 0

// The lanes that hold the largest (c, then l) key of the warp.
__device__ __forceinline__ uint32_t best_lanes(uint64_t c, uint32_t l) {
  const uint32_t hi = (uint32_t)(c >> 32), lo = (uint32_t)c;
  const uint32_t mh = __reduce_max_sync(kFull, hi);
  const uint32_t ml = __reduce_max_sync(kFull, hi == mh ? lo : 0u);
  const bool in = hi == mh && lo == ml;
  const uint32_t mk = __reduce_max_sync(kFull, in ? l : 0u);
  return __ballot_sync(kFull, in && l == mk);
}

// Lane j < top_k gets the j-th choice; called by the whole warp.  unsure: the precision could
// not order two scores.
template <class S, int NV, class TL>
__device__ __noinline__ int rank_again(const TL* row, const RouteArgs& a, bool* unsure) {
  const int lane = threadIdx.x & 31;
  const int size = a.size, grp = lane / a.lpg, in = (lane % a.lpg) * NV;
  const int base = grp * size + in;
  const int cnt = grp < a.n_group ? max(0, min(NV, size - in)) : 0;
  uint64_t c[NV];
  uint32_t lk[NV];
  bool doubt = false;

  float m = -INFINITY;
  for (int i = 0; i < cnt; ++i) m = fmaxf(m, clean_logit(load1(row + base + i)));
  m = warp_max(m);
  typename S::V den = S::of(0.f);  // the softmax's denominator
  if (a.score == MOE_SCORE_SOFTMAX) {
    for (int i = 0; i < cnt; ++i) {
      const float l = clean_logit(load1(row + base + i));
      if (l > -INFINITY) den = S::plus(den, S::exp_diff(l, m));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) den = S::plus(den, S::shfl(den, off));
  }
  auto score_of = [&](float l) {
    if (a.score == MOE_SCORE_SOFTMAX) return S::quotient(S::exp_diff(l, m), den);
    const typename S::V e = S::exp_diff(-fabsf(l), 0.f);
    return S::quotient(l < 0.f ? e : S::of(1.f), S::plus(S::of(1.f), e));
  };
  const bool by_logit = a.bias == nullptr;  // the logits' order is the scores'
#pragma unroll 1
  for (int i = 0; i < NV; ++i) {
    c[i] = 0;
    lk[i] = 0;
    if (i >= cnt) continue;
    float l, b;
    expert_inputs(row, a.bias, base + i, l, b);
    if (l == -INFINITY) {
      c[i] = kMasked64;
      continue;
    }
    lk[i] = order_key(l);
    if (by_logit)
      c[i] = (uint64_t)lk[i] << 32;
    else
      c[i] = S::key(b == INFINITY ? S::of(b) : S::plus(score_of(l), S::of(b)));
  }
  if (a.n_group > 1) {
    uint64_t top = 0, second = 0;
#pragma unroll 1
    for (int i = 0; i < NV; ++i) {
      if (c[i] > top) {
        second = top;
        top = c[i];
      } else if (c[i] > second) {
        second = c[i];
      }
    }
    for (int off = 1; off < a.lpg; off <<= 1) {
      const uint64_t t = __shfl_xor_sync(kFull, top, off), u = __shfl_xor_sync(kFull, second, off);
      second = max(min(top, t), max(second, u));
      top = max(top, t);
    }
    uint64_t score = top;
    const bool sums = a.group_top == 2;
    if (sums && top > kMasked64) {
      auto value = [&](uint64_t k) { return by_logit ? score_of(key_value((uint32_t)(k >> 32))) : S::value(k); };
      typename S::V x = value(top);
      if (second > kMasked64 && top != S::key(S::of(INFINITY))) x = S::plus(x, value(second));
      score = S::key(x);
    }
    int rank = 0;
#pragma unroll 1
    for (int g = 0; g < a.n_group; ++g) {
      const uint64_t o = __shfl_sync(kFull, score, g * a.lpg);
      rank += o > score || (o == score && g < grp);
    }
    const bool keep = grp < a.n_group && rank < a.topk_group;
    if (a.topk_group < a.n_group) {
      // the last group kept and the first left out
      const int last = __ffs(__ballot_sync(kFull, grp < a.n_group && rank == a.topk_group - 1)) - 1;
      const int next = __ffs(__ballot_sync(kFull, grp < a.n_group && rank == a.topk_group)) - 1;
      const uint64_t x = __shfl_sync(kFull, score, last), y = __shfl_sync(kFull, score, next);
      doubt = y > kMasked64 && (sums || !by_logit) && S::near(x, y);
    }
    if (!keep) {
#pragma unroll 1
      for (int i = 0; i < NV; ++i) c[i] = 0;
    }
  }
  // top_k rounds, then on until the rest is surely below the last choice (one that is equal to it does
  // not vouch for what comes after)
  int mine = 0, prev_id = 0;
  uint64_t prev = 0, last = 0;
#pragma unroll 1
  for (int r = 0;; ++r) {
    uint64_t bc = 0;
    uint32_t bl = 0;
    int at = 0;
#pragma unroll 1
    for (int i = 0; i < NV; ++i)
      if (c[i] > bc || (c[i] == bc && lk[i] > bl)) {
        bc = c[i];
        bl = lk[i];
        at = i;
      }
    const int w = __ffs(best_lanes(bc, bl)) - 1;
    const uint64_t top = __shfl_sync(kFull, bc, w);
    const int id = __shfl_sync(kFull, base + at, w);
    if (r > 0 && top > kMasked64 && !by_logit && S::near(prev, top)) {
      float lx, bx, ly, by;
      expert_inputs(row, a.bias, prev_id, lx, bx);
      expert_inputs(row, a.bias, id, ly, by);
      doubt |= !(lx == ly && bx == by);
    }
    if (r >= a.top_k && (doubt || by_logit || top <= kMasked64 || !S::near(last, top))) break;
    if (lane == w) c[at] = 0;
    if (lane == w) lk[at] = 0;
    if (lane == r && r < a.top_k) mine = id;
    if (r == a.top_k - 1) last = top;
    prev = top;
    prev_id = id;
  }
  *unsure = doubt;
  return mine;
}

// The softmax's denominator over the warp's logits (cnt of them at p in this lane): its terms are
// within 1 ulp, and their sum adds nothing.
template <class TL>
__device__ __noinline__ FF sum_ff(const TL* p, int cnt, float m) {
  FF sum{0.f, 0.f};
  for (int i = 0; i < cnt; ++i) {
    const float x = clean_logit(load1(p + i));
    if (x > -INFINITY) sum = add(sum, {expf(x - m), 0.f});
  }
  for (int off = 16; off > 0; off >>= 1) sum = add(sum, PairScores::shfl(sum, off));
  return sum;
}
__device__ __forceinline__ FF sigmoid_ff(float l) {
  const FF e = exp_ff({-fabsf(l), 0.f});
  return div(l < 0.f ? e : FF{1.f, 0.f}, add({1.f, 0.f}, e));
}

// Lane i < n has candidate id: lane j gets the j-th of them (n <= 32) by the scores in pairs of
// floats.  m, den: the row's softmax, den within 2^-22 (an error in it moves all scores of the row
// by one factor, so it counts by the scores' difference).
template <class TL>
__device__ __noinline__ int rank_candidates(const TL* row, const RouteArgs& a, int id, int n, float m, FF den,
                                            bool* unsure) {
  const int lane = threadIdx.x & 31;
  float l = -INFINITY, b = 0.f;
  if (lane < n) expert_inputs(row, a.bias, id, l, b);
  uint64_t c = 0;
  FF s{0.f, 0.f};
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  if (a.bias == nullptr) {
    c = (uint64_t)order_key(l) << 32;
  } else {
    s = softmax ? div(exp_ff(two_sum(l, -m)), den) : sigmoid_ff(l);
    c = l == -INFINITY ? kMasked64 : PairScores::key(b == INFINITY ? FF{b, 0.f} : add(s, {b, 0.f}));
  }
  int rank = 0;
  bool doubt = false;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const uint64_t o = __shfl_sync(kFull, c, j);
    const float ol = __shfl_sync(kFull, l, j), ob = __shfl_sync(kFull, b, j);
    const int oid = __shfl_sync(kFull, id, j);
    const bool same = ol == l && ob == b;  // equal scores: the lower index first
    rank += same ? oid < id : o > c;
    const float apart = softmax ? 0x1p-22f * fabsf(__shfl_sync(kFull, s.h, j) - s.h) : 0.f;
    doubt |= a.bias != nullptr && !same && lane < n && min(o, c) > kMasked64 &&
             PairScores::near(max(o, c), min(o, c), apart);
  }
  *unsure = __any_sync(kFull, doubt);
  int got = 0;
  for (int j = 0; j < n; ++j) {
    const int at = __shfl_sync(kFull, rank, j), v = __shfl_sync(kFull, id, j);
    if (lane == at) got = v;
  }
  return got;
}

// ------------------------------------------------------------------ forward
__device__ __forceinline__ void order2(uint32_t& a, uint32_t& b) {
  const uint32_t x = max(a, b), y = min(a, b);
  a = x;
  b = y;
}
// Batcher's odd-even merge sort, descending.
template <int NV>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[NV]) {
#pragma unroll
  for (int p = 1; p < NV; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j <= NV - 1 - k; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < NV && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order2(key[i + j], key[i + j + k]);
}

// Distances below which two ranking scores may be in the wrong order.  fast_exp(-x) is within
// (2 + 1.2 x) 2^-23 of its value.  Sigmoid: that moves s by at most 0.65 2^-23, the sum and the
// division (2 roundings) by 2.5 2^-23: two scores are within 2^-20.3.  Softmax: a score's own exponential
// and division give 2^-21; the denominator moves all scores of a row by one common factor, within
// 2^-18.2 (its terms' errors weighed by the terms, whose mean x is at most ln E, and up to 69
// additions): 2^-17.6 for two.  Adding the bias rounds by 2^-24 |c| and cutting the places off the
// keys by NV 2^-23 |c| (cut).
struct Doubt {
  bool by_logit, exact16;  // ranked by logits; they fit the keys whole (16-bit types)
  float tol0, cut;
  // x >= y are two keys (without places): may their experts be in the other order?
  __device__ __forceinline__ bool of(uint32_t kx, uint32_t ky, uint32_t none) const {
    if (ky <= none) return false;
    if (by_logit) return !exact16 && kx == ky;
    const float x = key_value(kx), y = key_value(ky);
    return !(x - y > tol0 + cut * (fabsf(x) + fabsf(y)));
  }
  // the same for the scores of the last group kept and the best left out, err from the cuts
  __device__ __forceinline__ bool groups(uint32_t kx, uint32_t ky, float err) const {
    const float x = key_value(kx), y = key_value(ky);
    float tol = 2.f * (tol0 + err) + 0x1p-22f * (fabsf(x) + fabsf(y));
    // without a bias the errors are relative too (the exponential's at most (2 + 1.2 88) 2^-23, the
    // cut logits' err): sums of small scores are told apart by their own size.  An exponential below
    // 2^-126 counts as 0, which takes up to 2^-125 from a sum of two, and one last place of a subnormal
    // product with 1 / den is 2^-149: within 2^-124 for two sums.
    if (by_logit) tol = fminf(tol, (0x1p-15f + 8.f * cut) * (x + y) + 2.f * err * (x + y) + 0x1p-124f);
    return !(x - y > tol);
  }
};

// A score for ranking alone, by the fast exponential and division.
__device__ __forceinline__ float rank_score(float x, bool softmax, float m, float rden) {
  const float e = fast_exp(softmax ? x - m : -fabsf(x));
  return softmax ? e * rden : (x < 0.f ? e : 1.0f) * fast_rcp(1.0f + e);
}

// A group's score as an ordered key, from its two best keys (`none`: a masked one); err: how far the
// places cut off the keys may have moved it.
__device__ __forceinline__ uint32_t group_score(uint32_t top, uint32_t second, uint32_t none, bool sums, bool by_logit,
                                                bool softmax, float m, float rden, float cut, float& err) {
  err = 0.f;
  if (top <= none) return top;  // (a masked group keeps the masked key)
  if (!sums) {
    if (!by_logit) err = cut * fabsf(key_value(top));
    return top;
  }
  float x = key_value(top), y = second > none ? key_value(second) : 0.f;
  err = cut * (fabsf(x) + fabsf(y));
  if (by_logit) {
    // the cut logits' distance moves a sigmoid by less than 0.3 of its relative size, a softmax
    // numerator by all of it
    x = rank_score(x, softmax, m, rden);
    y = second > none ? rank_score(y, softmax, m, rden) : 0.f;
  }
  return order_key(x + y);
}

// The weight (before the scale) of a lane's choice with logit lj (-inf: masked, or no choice); m and
// den: the row's softmax.  Called by the whole warp.
__device__ __forceinline__ float choice_weight(const RouteArgs& a, float lj, float m, float den) {
  const bool live = lj > -INFINITY, softmax = a.score == MOE_SCORE_SOFTMAX;
  if (!a.renorm) return !live ? 0.f : softmax ? __fdividef(exp_below(lj, m), den) : sigmoid32(lj);
  // s_j / sum s is the same for scores scaled by one factor: softmax numerators relative to the
  // largest chosen, sigmoid scores by e^-m (m = the largest chosen logit when all are negative)
  // so that none underflows
  const float top = warp_max(lj);
  float s = 0.f;
  if (live) {
    if (softmax)
      s = exp_below(lj, top);
    else
      s = top < 0.f ? __fdividef(exp_below(lj, top), 1.0f + expf(lj)) : sigmoid32(lj);
  }
  const float sum = warp_sum(s);
  return sum > 0.f ? __fdividef(s, sum) : 0.f;  // (the sum lies in [1/2, 32])
}

// One token by one warp.  NV: experts held by a lane, a power of two.  TL: type of the logits.
template <int NV, class TL>
__global__ void __launch_bounds__(kWarpsPerBlock * 32)
    route_grouped_kernel(const RouteArgs a, int32_t* __restrict__ topk_ids, float* __restrict__ topk_weights) {
  constexpr uint32_t kPlace = NV - 1;             // the key bits that hold NV - 1 - place
  constexpr uint32_t kNone = kMaskedKey & ~kPlace;  // a masked expert's key without its place
  constexpr bool kSorted = NV <= 16;              // (longer lists are searched again each round)
  const int t = blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int lane = threadIdx.x & 31;
  const TL* row = static_cast<const TL*>(a.logits) + (size_t)t * a.E;
  const bool by_logit = a.bias == nullptr, softmax = a.score == MOE_SCORE_SOFTMAX;
  const int size = a.size, grp = lane / a.lpg, in = (lane % a.lpg) * NV;
  const int base = grp * size + in;
  const int cnt = grp < a.n_group ? min(NV, size - in) : 0;  // (may be negative: none)

  float l[NV];
  load_lane<NV>(row + base, cnt, size, l);
  uint32_t key[NV];
  float b[NV];
  if (!by_logit) load_lane<NV>(a.bias + base, cnt, size, b);
  // the row's largest logit and the softmax's denominator, where a score is needed
  float m = 0.f, den = 1.f;
  if (softmax && (!by_logit || !a.renorm || (a.n_group > 1 && a.group_top == 2))) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) m = fmaxf(m, clean_logit(l[i]));
    m = warp_max(m);
    den = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float x = clean_logit(l[i]);
      if (x > -INFINITY) den += __expf(x - m);
    }
    den = warp_sum(den);
  }
  const float rden = __fdividef(1.0f, den);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const float x = clean_logit(l[i]);
    uint32_t k;
    if (by_logit) {
      k = order_key(x);
    } else {
      const bool gone = x == -INFINITY || b[i] != b[i] || b[i] == -INFINITY;
      k = gone ? kMaskedKey : order_key(rank_score(x, softmax, m, rden) + b[i]);
    }
    key[i] = i < cnt ? (k & ~kPlace) | (kPlace - i) : 0u;
  }
  if (kSorted) sort_keys(key);

  const Doubt doubt{by_logit, sizeof(TL) == 2, softmax ? 0x1p-17f : 0x1p-20f, (NV + 2) * 0x1p-23f};
  bool unsure = false;

  if (a.n_group > 1) {
    uint32_t top = 0, second = 0;
    const bool exact = by_logit && a.group_top == 1;  // whole logits: nothing cut off
    if (exact) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i < cnt) top = max(top, order_key(clean_logit(l[i])));
    } else if (kSorted) {
      top = key[0] & ~kPlace;
      second = NV > 1 ? key[NV > 1 ? 1 : 0] & ~kPlace : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t k = key[i] & ~kPlace;
        second = max(second, min(top, k));
        top = max(top, k);
      }
    }
    for (int off = 1; off < a.lpg; off <<= 1) {
      const uint32_t x = __shfl_xor_sync(kFull, top, off), y = __shfl_xor_sync(kFull, second, off);
      second = max(min(top, x), max(second, y));
      top = max(top, x);
    }
    float err;
    const uint32_t score = group_score(top, second, kNone, a.group_top == 2, by_logit, softmax, m, rden, doubt.cut, err);
    int rank = 0;
#pragma unroll 4
    for (int g = 0; g < a.n_group; ++g) {
      const uint32_t o = __shfl_sync(kFull, score, g * a.lpg);
      rank += o > score || (o == score && g < grp);
    }
    const bool keep = rank < a.topk_group && grp < a.n_group;
    const uint32_t last = __reduce_min_sync(kFull, keep ? score : kFull);
    const uint32_t left = __reduce_max_sync(kFull, keep || grp >= a.n_group ? 0u : score);  // 0: none left out
    if (left > kNone && !exact) unsure = doubt.groups(last, left, warp_max(err));
    if (!keep) {
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = 0;
    }
  }

  // top_k rounds, then one for the best expert left out; where some order is in doubt (near), more
  // until the rest is surely below the last choice.  Lane r keeps the r-th.
  int my_id = 0;
  uint32_t prev_key = 0, last_key = 0;
  int prev_id = 0, r = 0;
  bool near = false;
  auto head = [&]() {
    if (kSorted) return key[0];
    uint32_t h = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) h = max(h, key[i]);
    return h;
  };
  uint32_t h = head();
  auto in_doubt = [&](uint32_t kx, uint32_t ky) { return doubt.of(kx, ky, kNone); };
#pragma unroll 1
  for (;; ++r) {
    const uint32_t top = __reduce_max_sync(kFull, h & ~kPlace);
    if (r >= a.top_k) {
      near |= in_doubt(prev_key, top);
      if (!near || !in_doubt(last_key, top)) break;
      if (r == 32) {  // more candidates than lanes
        unsure = true;
        break;
      }
    }
    const int w = __ffs(__ballot_sync(kFull, (h & ~kPlace) == top)) - 1;
    const int id = __shfl_sync(kFull, base + (int)(kPlace - (h & kPlace)), w);
    if (lane == w) {
      if (kSorted) {
#pragma unroll
        for (int i = 0; i + 1 < NV; ++i) key[i] = key[i + 1];
        key[NV - 1] = 0;
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (key[i] == h) key[i] = 0;
      }
      h = head();
    }
    if (r > 0 && !near && in_doubt(prev_key, top)) {
      // equal logit and bias: equal scores, and the lower index came first
      float lx, bx, ly, by;
      expert_inputs(row, a.bias, prev_id, lx, bx);
      expert_inputs(row, a.bias, id, ly, by);
      near = !(lx == ly && bx == by);
    }
    prev_key = top;
    prev_id = id;
    if (r == a.top_k - 1) last_key = top;
    if (lane == r) my_id = id;
  }
  if (near && !unsure) {
    // the r candidates, one a lane, ranked by their exact scores
    my_id = rank_candidates(row, a, my_id, r, m, softmax && !by_logit ? sum_ff(row + base, cnt, m) : FF{1.f, 0.f},
                            &unsure);
  }
  if (unsure) {
    my_id = rank_again<PairScores, NV, TL>(row, a, &unsure);
    if (unsure) my_id = rank_again<DoubleScores, NV, TL>(row, a, &unsure);
  }

  // weights: lane j has the j-th choice
  float lj = -INFINITY, bj = 0.f;
  if (lane < a.top_k) expert_inputs(row, a.bias, my_id, lj, bj);
  if (softmax && !a.renorm) {  // the denominator again, by the accurate exponential
    den = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float x = clean_logit(l[i]);
      if (x > -INFINITY) den += expf(x - m);
    }
    den = warp_sum(den);
  }
  const float w = choice_weight(a, lj, m, den);
  if (lane < a.top_k) {
    topk_ids[(size_t)t * a.top_k + lane] = my_id;
    topk_weights[(size_t)t * a.top_k + lane] = w * a.scale;
  }
}

// Up to 16 choices among up to 8 experts a lane, one token by one warp, without rounds: every lane
// sorts its keys, and five butterfly steps merge the lists of two lanes into the best 8 (or 16) of
// both, so that all lanes end with the chosen ones in order.  A merge of two sorted lists of 8 takes 8
// shuffles, 8 maxima (of one list against the other reversed, which leaves the best 8 as a
// bitonic sequence) and 12 comparators.  The keys carry the expert's place in the warp in their low
// bits (8 of them for 256 experts), so a key names its expert; the cut makes a few tokens in a
// hundred doubtful, whose candidates are ranked exactly.  Against rounds of redux.sync (the kernel
// above), in a graph, 256 experts, 4 of 8 groups, bias: one token 4.2 -> 3.0 us, 16384 tokens 33 ->
// 23.5 us (0.8 TB/s).  It is bound by the integer pipe that does the minima and maxima: two tokens
// a warp, 16 lanes each, took a quarter fewer instructions and the same time, and four tokens of
// 32 experts a lane twice the time.
// a[0..N) is bitonic: sorted descending
template <int N, int M>
__device__ __forceinline__ void bitonic_sort(uint32_t (&a)[M]) {
#pragma unroll
  for (int k = N / 2; k >= 1; k /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & k) == 0) order2(a[i], a[i + k]);
}
// The best KL of the warp's lists of LEN sorted keys; OFF: lanes merged so far.
template <int LEN, int OFF, int KL>
__device__ __forceinline__ void merge_lists(uint32_t (&a)[KL]) {
  if constexpr (OFF < 32) {
    uint32_t o[LEN];
#pragma unroll
    for (int i = 0; i < LEN; ++i) o[i] = __shfl_xor_sync(kFull, a[i], OFF);
    if constexpr (LEN < KL) {
#pragma unroll
      for (int i = 0; i < LEN; ++i) a[LEN + i] = o[LEN - 1 - i];
      bitonic_sort<2 * LEN>(a);
      merge_lists<2 * LEN, 2 * OFF>(a);
    } else {
#pragma unroll
      for (int i = 0; i < KL; ++i) a[i] = max(a[i], o[KL - 1 - i]);
      bitonic_sort<KL>(a);
      merge_lists<KL, 2 * OFF>(a);
    }
  }
}

// KL: 8 or 16, at least top_k.
template <int NV, int KL, class TL>
__global__ void __launch_bounds__(kWarpsPerBlock * 32)
    route_grouped_merge_kernel(const RouteArgs a, int32_t* __restrict__ topk_ids, float* __restrict__ topk_weights) {
  constexpr uint32_t kPlace = 32 * NV - 1;  // the key bits that hold kPlace - (place in the warp)
  constexpr uint32_t kNone = kMaskedKey & ~kPlace;
  const int t = blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int lane = threadIdx.x & 31;
  const TL* row = static_cast<const TL*>(a.logits) + (size_t)t * a.E;
  const bool by_logit = a.bias == nullptr, softmax = a.score == MOE_SCORE_SOFTMAX;
  const int lpg = a.lpg, size = a.size, lane_shift = __ffs(lpg) - 1;
  const int grp = lane >> lane_shift, in = (lane & (lpg - 1)) * NV;
  const int base = grp * size + in;
  const int cnt = grp < a.n_group ? min(NV, size - in) : 0;  // (may be negative: none)

  float m = 0.f, den = 1.f;
  uint32_t key[NV];
  {
    float l[NV];
    load_lane<NV>(row + base, cnt, size, l);
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = clean_logit(l[i]);
    // the row's largest logit and the softmax's denominator, where a score is needed
    if (softmax && (!by_logit || !a.renorm || (a.n_group > 1 && a.group_top == 2))) {
      m = -INFINITY;
#pragma unroll
      for (int i = 0; i < NV; ++i) m = fmaxf(m, l[i]);
      m = warp_max(m);
      den = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (l[i] > -INFINITY) den += expf(l[i] - m);
      den = warp_sum(den);
    }
    if (by_logit) {
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = order_key(l[i]);
    } else {
      float b[NV];
      load_lane<NV>(a.bias + base, cnt, size, b);
      const float rden = __fdividef(1.0f, den);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        // (a NaN or -inf bias masks: the sum is then NaN or -inf too)
        const float c = rank_score(l[i], softmax, m, rden) + b[i];
        key[i] = l[i] > -INFINITY && c > -INFINITY ? order_key(c) : kMaskedKey;
      }
    }
    if (cnt < NV) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i >= cnt) key[i] = 0;
    }
  }
  Doubt doubt{by_logit, sizeof(TL) == 2, softmax ? 0x1p-17f : 0x1p-20f, 0x1p-22f};
  bool unsure = false, dropped = false;

  if (a.n_group > 1) {
    uint32_t top = 0, second = 0;  // whole keys: the groups' order is hardly ever in doubt
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      second = max(second, min(top, key[i]));
      top = max(top, key[i]);
    }
    for (int off = 1; off < lpg; off <<= 1) {
      const uint32_t x = __shfl_xor_sync(kFull, top, off), y = __shfl_xor_sync(kFull, second, off);
      second = max(min(top, x), max(second, y));
      top = max(top, x);
    }
    float err;
    const uint32_t score = group_score(top, second, kMaskedKey, a.group_top == 2, by_logit, softmax, m,
                                       __fdividef(1.0f, den), doubt.cut, err);
    int rank = 0;
#pragma unroll 4
    for (int g = 0; g < a.n_group; ++g) {
      const uint32_t o = __shfl_sync(kFull, score, g << lane_shift);
      rank += o > score || (o == score && g < grp);
    }
    const bool in_use = grp < a.n_group;
    bool keep = in_use && rank < a.topk_group;
    const uint32_t last = __reduce_min_sync(kFull, keep ? score : kFull);
    const uint32_t left = __reduce_max_sync(kFull, keep || !in_use ? 0u : score);  // 0: none left out
    if (left > kMaskedKey && !(by_logit && a.group_top == 1)) {
      err = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(err)));
      if (doubt.groups(last, left, err)) {
        // Which of two groups?  Exactly, if only they are in doubt, from their group_top best experts
        // if these are surely the best: one expert a lane, 0 and 1 of the last group kept, 2 and 3
        // of the first left out.
        const uint32_t above = __reduce_min_sync(kFull, in_use && rank < a.topk_group - 1 ? score : kFull);
        const uint32_t below = __reduce_max_sync(kFull, in_use && rank > a.topk_group ? score : 0u);
        unsure = (above != kFull && doubt.groups(above, left, err)) ||
                 (below > kMaskedKey && doubt.groups(last, below, err));
        const int ga = __shfl_sync(kFull, grp, __ffs(__ballot_sync(kFull, in_use && rank == a.topk_group - 1)) - 1);
        const int gb = __shfl_sync(kFull, grp, __ffs(__ballot_sync(kFull, in_use && rank == a.topk_group)) - 1);
        int id = -1;
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
          const int want = g ? gb : ga;
          uint32_t prev = 0;
          int first = -1;
#pragma unroll 1
          for (int j = 0; j <= a.group_top; ++j) {  // (the last of them: the best expert that does not count)
            uint32_t v = 0;
            int at = -1;
#pragma unroll
            for (int i = 0; i < NV; ++i)
              if (grp == want && (j == 0 || key[i] < prev || (key[i] == prev && base + i > first)) && key[i] > v) {
                v = key[i];
                at = base + i;
              }
            const uint32_t best_key = __reduce_max_sync(kFull, v);
            const int w = __ffs(__ballot_sync(kFull, v == best_key)) - 1, e = __shfl_sync(kFull, at, w);
            if (j == a.group_top)
              unsure |= !by_logit && best_key > kMaskedKey && doubt.of(prev, best_key, kMaskedKey);
            else if (lane == 2 * g + j && best_key > kMaskedKey)
              id = e;
            prev = best_key;
            first = e;
          }
        }
        if (!unsure) {
          const bool divide = softmax && !by_logit;  // (else a softmax's numerators order like its scores)
          const FF sum = divide ? sum_ff(row + base, cnt, m) : FF{1.f, 0.f};
          FF c{0.f, 0.f};
          // (a lane without an expert, of a group with fewer usable ones than group_top, has a logit that no
          // expert here has: it equals only another of its kind); part: the scores without the biases
          float x = -INFINITY, b = 0.f, part = 0.f;
          if (id >= 0) {
            expert_inputs(row, a.bias, id, x, b);
            c = softmax ? exp_ff(two_sum(x, -m)) : sigmoid_ff(x);
            if (divide) c = div(c, sum);
            part = c.h;
            c = b == INFINITY ? FF{b, 0.f} : add(c, {b, 0.f});
          }
          part += __shfl_xor_sync(kFull, part, 1);
          const float apart = divide ? 0x1p-22f * fabsf(__shfl_sync(kFull, part, 0) - __shfl_sync(kFull, part, 2)) : 0.f;
          const FF o = PairScores::shfl(c, 1);
          c = c.h == INFINITY || o.h == INFINITY ? FF{fmaxf(c.h, o.h), 0.f} : add(c, o);
          const uint64_t sa = __shfl_sync(kFull, PairScores::key(c), 0), sb = __shfl_sync(kFull, PairScores::key(c), 2);
          // (equal logits and biases: equal scores, and the lower group was kept)
          const float x2 = __shfl_down_sync(kFull, x, 2), b2 = __shfl_down_sync(kFull, b, 2);
          const bool same = __all_sync(kFull, lane >= 2 || (x == x2 && b == b2));
          unsure = !same && PairScores::near(max(sa, sb), min(sa, sb), apart);
          if (!same && sb > sa) keep = (keep && grp != ga) || (in_use && grp == gb);
        }
      }
    }
    dropped = !keep;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) key[i] = key[i] && !dropped ? (key[i] & ~kPlace) | (kPlace - (lane * NV + i)) : 0u;
  doubt.cut = (32 * NV + 2) * 0x1p-23f;
  sort_keys(key);

  uint32_t best[KL];
#pragma unroll
  for (int i = 0; i < KL; ++i) best[i] = i < NV ? key[i < NV ? i : 0] : 0u;
  merge_lists<NV, 1>(best);

  // lane r holds the r-th best; the first left out (none: 0) after them
  auto next_below = [&](uint32_t bound) {  // the warp's largest key below bound
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) v = max(v, key[i] < bound ? key[i] : 0u);
    return __reduce_max_sync(kFull, v);
  };
  uint32_t mine = 0;
  {
    uint32_t h[KL];
#pragma unroll
    for (int i = 0; i < KL; ++i) h[i] = best[i];
#pragma unroll
    for (int n = KL / 2, bit = 1; n >= 1; n /= 2, bit *= 2)
#pragma unroll
      for (int i = 0; i < n; ++i) h[i] = lane & bit ? h[2 * i + 1] : h[2 * i];
    if (lane < KL) mine = h[0];
  }
  if (a.top_k == KL) {
    const uint32_t v = next_below(best[KL - 1]);
    if (lane == KL) mine = v;
  }
  auto expert_of = [&](uint32_t k) {
    const int pos = (int)(kPlace - (k & kPlace)), ln = pos / NV;
    return k ? (ln >> lane_shift) * size + (ln & (lpg - 1)) * NV + pos % NV : 0;
  };
  int my_id = expert_of(mine);
  float lj = -INFINITY, bj = 0.f;
  if (lane <= a.top_k && mine) expert_inputs(row, a.bias, my_id, lj, bj);
  {
    // doubt between neighbours, unless they are equal in logit and bias
    const uint32_t next = __shfl_down_sync(kFull, mine, 1) & ~kPlace;
    const float ln = __shfl_down_sync(kFull, lj, 1), bn = __shfl_down_sync(kFull, bj, 1);
    const bool close = lane < a.top_k && doubt.of(mine & ~kPlace, next, kNone), equal = ln == lj && bn == bj;
    bool near = __any_sync(kFull, close && !equal);
    if (!near && __any_sync(kFull, close && lane == a.top_k - 1)) {
      // the first left out equals the last choice: it does not vouch for what comes after
      const uint32_t last = __shfl_sync(kFull, mine, a.top_k - 1);
      const float ll = __shfl_sync(kFull, lj, a.top_k - 1), bl = __shfl_sync(kFull, bj, a.top_k - 1);
      uint32_t low = __shfl_sync(kFull, mine, a.top_k);
      while (!near) {
        low = next_below(low);
        if (!doubt.of(last & ~kPlace, low & ~kPlace, kNone)) break;
        float x, b;
        expert_inputs(row, a.bias, expert_of(low), x, b);
        near = !(x == ll && b == bl);
      }
    }
    if (near || unsure) {
      if (!unsure) {
        // the candidates, one a lane: all that are not surely below the last choice
        const uint32_t last = __shfl_sync(kFull, mine, a.top_k - 1);
        uint32_t low = last;
        int n = a.top_k;
        while (true) {
          low = next_below(low);
          if (!doubt.of(last & ~kPlace, low & ~kPlace, kNone)) break;
          if (n == 32) {
            unsure = true;
            break;
          }
          if (lane == n) my_id = expert_of(low);
          ++n;
        }
        if (!unsure)
          my_id = rank_candidates(row, a, my_id, n, m,
                                  softmax && !by_logit ? sum_ff(row + base, cnt, m) : FF{1.f, 0.f}, &unsure);
      }
      if (unsure) my_id = rank_again<PairScores, NV, TL>(row, a, &unsure);
      if (unsure) my_id = rank_again<DoubleScores, NV, TL>(row, a, &unsure);
      lj = -INFINITY;
      if (lane < a.top_k) expert_inputs(row, a.bias, my_id, lj, bj);
    }
  }
  if (lane >= a.top_k) lj = -INFINITY;
  const float w = choice_weight(a, lj, m, den);
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
      float b;
      expert_inputs(row, a.bias, id, lj, b);  // (the bias only masks here)
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
        s = exp_below(lj, top);
      } else {
        s = top < 0.f ? __fdividef(exp_below(lj, top), 1.0f + expf(lj)) : sigmoid32(lj);
        f = sigmoid32(-lj);  // 1 - s without the cancellation
      }
    }
    const float sum = warp_sum(s);
    const float p = sum > 0.f ? __fdividef(s, sum) : 0.f;
    const float mean = warp_sum(p * dw);
    d = p * f * (dw - mean);
  } else if (a.score == MOE_SCORE_SIGMOID) {
    if (live) d = dw * sigmoid32(lj) * sigmoid32(-lj);
  }
  if (!a.renorm && a.score == MOE_SCORE_SOFTMAX) {
    float s[NV];
    load_lane<NV>(row + lane * NV, a.E - lane * NV, a.E, s);
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = clean_logit(s[i]);
      m = fmaxf(m, s[i]);
    }
    m = warp_max(m);
    float den = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = exp_below(s[i], m);  // (0 for a masked logit)
      den += s[i];
    }
    den = warp_sum(den);
    d = live ? dw * __fdividef(exp_below(lj, m), den) : 0.f;  // g_j s_j
    const float dot = warp_sum(d), rden = den > 0.f ? __fdividef(-dot, den) : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] *= rden;
    if constexpr (NV >= 4) {
#pragma unroll
      for (int i = 0; i < NV; i += 4)
        *reinterpret_cast<float4*>(buf + lane * NV + i) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) buf[lane * NV + i] = s[i];
    }
  } else {
    for (int i = lane * 4; i < 32 * NV; i += 128) *reinterpret_cast<float4*>(buf + i) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
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

// Lanes of a group, and the experts a lane then holds (at most 64: 17 groups of 60 on a lane each).
int lanes_per_group(int n_group) {
  int lpg = 32;
  while (lpg * n_group > 32) lpg /= 2;
  return lpg;
}

template <class F>
void for_nv(int nv, F f) {
  if (nv <= 1) return f(std::integral_constant<int, 1>());
  if (nv <= 2) return f(std::integral_constant<int, 2>());
  if (nv <= 4) return f(std::integral_constant<int, 4>());
  if (nv <= 8) return f(std::integral_constant<int, 8>());
  if (nv <= 16) return f(std::integral_constant<int, 16>());
  if (nv <= 32) return f(std::integral_constant<int, 32>());
  return f(std::integral_constant<int, 64>());
}

moe_status_t check_route(moe_dtype_t dt, int T, int E, int top_k, const moe_route_config* c) {
  MOE_CHECK_ARG(c && T >= 0 && T <= (1 << 30) && E >= 1 && E <= 1024 && top_k >= 1 && top_k <= 32);
  MOE_CHECK_ARG(c->n_group >= 1 && c->n_group <= 32 && E % c->n_group == 0);
  MOE_CHECK_ARG(c->topk_group >= 1 && c->topk_group <= c->n_group && top_k <= c->topk_group * (E / c->n_group));
  MOE_CHECK_ARG((c->group_top == 1 || c->group_top == 2) && c->group_top <= E / c->n_group);
  MOE_CHECK_ARG(c->score == MOE_SCORE_SOFTMAX || c->score == MOE_SCORE_SIGMOID);
  MOE_CHECK_ARG(c->scale - c->scale == 0.f);  // finite
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
  RouteArgs a{logits,          bias,           T,              E,               top_k,     cfg->score,
                    cfg->n_group, cfg->topk_group, cfg->group_top, cfg->renormalize, cfg->scale, E / cfg->n_group, 32};
  const dim3 grid((unsigned)((T + kWarpsPerBlock - 1) / kWarpsPerBlock)), block(kWarpsPerBlock * 32);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  a.lpg = lanes_per_group(cfg->n_group);
  const int size = E / cfg->n_group;
  auto with_type = [&](auto f) {
    if (logits_dtype == MOE_DT_FP32)
      f(float());
    else if (logits_dtype == MOE_DT_BF16)
      f(__nv_bfloat16());
    else
      f(__half());
  };
  for_nv((size + a.lpg - 1) / a.lpg, [&](auto n) {
    constexpr int NV = decltype(n)::value;
    with_type([&](auto tl) {
      if constexpr (NV <= 8) {
        if (top_k <= 8) {
          route_grouped_merge_kernel<NV, 8, decltype(tl)><<<grid, block, 0, s>>>(a, topk_ids, topk_weights);
          return;
        }
        if (top_k <= 16) {
          route_grouped_merge_kernel<NV, 16, decltype(tl)><<<grid, block, 0, s>>>(a, topk_ids, topk_weights);
          return;
        }
      }
      route_grouped_kernel<NV, decltype(tl)><<<grid, block, 0, s>>>(a, topk_ids, topk_weights);
    });
  });
  return launch_status();
}

extern "C" moe_status_t moe_route_grouped_backward(const float* dweights, const void* logits, moe_dtype_t logits_dtype,
                                                   const float* bias, const int32_t* topk_ids, int T, int E, int top_k,
                                                   const moe_route_config* cfg, void* dlogits, moe_stream_t stream) {
  const moe_status_t st = check_route(logits_dtype, T, E, top_k, cfg);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  MOE_CHECK_ARG(dweights && logits && topk_ids && dlogits);
  MOE_CHECK_ARG(aligned16(dweights) && aligned16(logits) && aligned16(bias) && aligned16(topk_ids) && aligned16(dlogits));
  const RouteArgs a{logits,          bias,           T,              E,               top_k,     cfg->score,
                    cfg->n_group, cfg->topk_group, cfg->group_top, cfg->renormalize, cfg->scale, E / cfg->n_group, 32};
  const dim3 grid((unsigned)((T + kWarpsPerBlock - 1) / kWarpsPerBlock)), block(kWarpsPerBlock * 32);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  for_nv((E + 31) / 32, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    if constexpr (NV > 32) return;  // E <= 1024
    else if (logits_dtype == MOE_DT_FP32)
      route_grouped_backward_kernel<NV, float>
          <<<grid, block, 0, s>>>(a, dweights, topk_ids, static_cast<float*>(dlogits));
    else if (logits_dtype == MOE_DT_BF16)
      route_grouped_backward_kernel<NV, __nv_bfloat16>
          <<<grid, block, 0, s>>>(a, dweights, topk_ids, static_cast<__nv_bfloat16*>(dlogits));
    else
      route_grouped_backward_kernel<NV, __half>
          <<<grid, block, 0, s>>>(a, dweights, topk_ids, static_cast<__half*>(dlogits));
  });
  return launch_status();
}
