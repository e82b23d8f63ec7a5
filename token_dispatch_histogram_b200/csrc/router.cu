// The router in front of the dispatch path: router logits to the K experts of
// each token and their gate weights, and the gradient of the weights.
//
// With x the logits of one token, s = softmax(x) or sigmoid(x) element by
// element, and b an optional bias per expert that balances the loads:
//   key_e = s_e + b_e, or x_e without a bias (the same order as s_e)
//   groups: the experts fall into n_group runs of E / n_group; a group's score
//     is its best key, or the sum of its best two (s_e without a bias); only
//     experts of the topk_group best groups are taken
//   ids = the K largest keys, descending; equal ones (of experts or of groups)
//     by ascending index
//   w_k = scale * s_k, or with renorm scale * s_k / sum_j s_j
// The bias moves the choice only; the weights and their gradient do not see it.
//
// Which of two experts comes first is decided by numbers that can lie closer
// than 32-bit scores tell apart, so keys and group scores are held in 64 bits.
// The weights are 32-bit ratios of exponentials of differences of logits: off by
// 2^-24 of the difference's size (its rounding) and a few units in the last place
// besides; without renorm a softmax divides by a sum of approximated exponentials
// (2^-22 of each), some units more.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

#include "common.cuh"

namespace ep {

constexpr int ROUTER_WARPS = 8;
constexpr int SMALL_E = 128;  // experts up to which eight lanes hold a token's logits

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// A logit as the definitions take it: -inf masks an expert, NaN counts as -inf
// and +inf as the largest finite value (both are flagged), so that every output
// is defined.
__device__ __forceinline__ float clean_logit(float x, bool& bad) {
  if (x <= FLT_MAX) return x;  // false for NaN and +inf
  bad = true;
  return x > 0.f ? FLT_MAX : -INFINITY;
}

// A NaN among the biases excludes its expert as -inf does: a key is never NaN.
__device__ __forceinline__ float clean_bias(float b) { return b == b ? b : -INFINITY; }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

__device__ __forceinline__ float warp_fmax(float v) {  // NaN on a lane counts as nothing
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float ex2_approx(float v) {  // 2^v, off by at most 2^-22 of it
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float rcp_approx(float v) {  // 1 / v, off by at most 2^-23 of it
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

constexpr float LOG2E = 1.44269504088896341f, LN2 = 0.693147180559945309f;

// e^v for v <= 0 to a few units in the last place: what the product with log2 e
// loses (found by the fused product) comes back as a factor.
__device__ __forceinline__ float exp_near(float v) {
  const float p = v * LOG2E, lost = fmaf(v, LOG2E, -p);
  return v < -87.f ? expf(v) : fmaf(ex2_approx(p) * LN2, lost, ex2_approx(p));
}

// s / sum_j s_j of a token's chosen logits, `width` lanes to a token (lane k < K
// holds x_k, the others -inf); 0 where all of them are -inf.  Both scores are e^x / (1 + e^x)
// or e^x over a common factor, so the ratio is taken of numbers scaled by the
// largest: no sum under- or overflows.
__device__ __forceinline__ float chosen_ratio(float x, bool sigmoid, int width) {
  float m = x;
  for (int d = width >> 1; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const bool none = m == -INFINITY;
  if (none) m = 0.f;
  float t;
  if (!sigmoid) {
    t = exp_near(x - m);
  } else {
    const float a = exp_near(-fabsf(x));  // s = 1 / (1 + a) or a / (1 + a)
    t = x >= 0.f ? 1.f : m >= 0.f ? a : exp_near(x - m);
    t = __fdividef(t, 1.f + a);
  }
  float sum = t;
  for (int d = width >> 1; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return none ? 0.f : __fdividef(t, sum);
}

__device__ __forceinline__ float sigmoid_f32(float x) {
  if (x >= 0.f) return 1.f / (1.f + expf(-x));
  const float e = expf(x);
  return e / (1.f + e);
}

struct RouterArgs {
  int64_t T, ld;
  int E, K, n_group, topk_group, group_top;
  bool sigmoid, renorm;
  float scale;
  int width;            // lanes to a token once its experts are chosen
  bool more;            // there are more than K experts to choose from
  int lanes_per_group;  // 32 / n_group, n_group rounded up to a power of two
  uint32_t group_inv;   // e * group_inv >> 21 == e / (E / n_group) for e < 1024
};

// One token by one warp, everything that decides held in 64 bits; key: E doubles
// of the warp's own.  Lane k < K returns the k-th expert.
template <typename V>
__device__ int select_exact(const RouterArgs& a, const V* __restrict__ row, const float* __restrict__ bias,
                            double* key) {
  const int lane = threadIdx.x & 31;
  const int len = a.E / a.n_group;
  const bool scores = bias != nullptr || (a.n_group > 1 && a.group_top == 2);
  bool bad = false;
  double m = -INFINITY, z = 0.0;
  if (scores && !a.sigmoid) {
    float mx = -INFINITY;
    for (int e = lane; e < a.E; e += 32) mx = fmaxf(mx, clean_logit(to_f32(row[e]), bad));
    m = warp_max(mx);
    for (int e = lane; e < a.E; e += 32) {
      const float x = clean_logit(to_f32(row[e]), bad);
      if (x != -INFINITY) z += exp((double)x - m);
    }
    z = warp_sum(z);
  }
  for (int e = lane; e < a.E; e += 32) {
    const double x = clean_logit(to_f32(row[e]), bad);
    double k = x;
    if (scores && x != -INFINITY) {
      if (!a.sigmoid)
        k = exp(x - m) / z;
      else if (x >= 0.0)
        k = 1.0 / (1.0 + exp(-x));
      else
        k = exp(x) / (1.0 + exp(x));
      if (bias) k += (double)clean_bias(bias[e]);
    }
    key[e] = k;
  }
  __syncwarp();
  uint32_t keep = 0xffffffffu;
  if (a.n_group > 1) {
    // lane g: the score of group g over its experts that are not masked
    double first = -INFINITY, second = -INFINITY;
    if (lane < a.n_group)
      for (int i = 0; i < len; ++i) {
        const double k = key[lane * len + i];
        if (k > first) {
          second = first;
          first = k;
        } else if (k > second) {
          second = k;
        }
      }
    double score = first;
    if (a.group_top == 2 && second != -INFINITY) score += second;
    int before = 0;
    for (int g = 0; g < a.n_group; ++g) {
      const double o = __shfl_sync(0xffffffffu, score, g);
      before += o > score || (o == score && g < lane);
    }
    keep = __ballot_sync(0xffffffffu, lane < a.n_group && before < a.topk_group);
    if (!bias && a.group_top == 2) {  // the groups were chosen by scores, the experts are by logits
      __syncwarp();
      for (int e = lane; e < a.E; e += 32) key[e] = clean_logit(to_f32(row[e]), bad);
      __syncwarp();
    }
  }
  int mine = 0;
  for (int k = 0; k < a.K; ++k) {
    double best = 0.0;
    int at = INT_MAX;
    for (int e = lane; e < a.E; e += 32) {
      const double v = key[e];
      if (isnan(v) || !(keep >> (a.n_group > 1 ? e / len : 0) & 1)) continue;  // taken, or of a group left out
      if (at == INT_MAX || v > best) {
        best = v;
        at = e;
      }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const double v = __shfl_xor_sync(0xffffffffu, best, d);
      const int o = __shfl_xor_sync(0xffffffffu, at, d);
      if (o != INT_MAX && (at == INT_MAX || v > best || (v == best && o < at))) {
        best = v;
        at = o;
      }
    }
    if (lane == k) mine = at;
    if (lane == (at & 31)) key[at] = NAN;
    __syncwarp();
  }
  return mine;
}

// Bounds of what the fast path's keys are off, from its steps: e^-x by ex2 of a
// rounded product (|x| 2^-24 and 2^-22 of itself), a sum, a quotient (2^-22), the
// bias added (2^-24 of the key).  Sigmoid: s (1 - s) |x| <= 0.23, so below 5e-7 of
// 1.  Softmax: a sum of up to 1024 terms besides (37 roundings of 2^-24), so below
// 4e-6 of s, and t e^-t <= 0.37 of 2^-23 for its own exponent.
__device__ __forceinline__ float key_error(bool sigmoid, float s, float key) {
  return (sigmoid ? 5e-7f : 1e-7f + 4e-6f * s) + 1.2e-7f * fabsf(key);
}

constexpr int HOISTED = 16;  // logits a lane up to which its biases stay in registers

// Lists of a warp: up to 64 candidates of the token at hand, in any order, and
// the first K + 1 of each token of a batch, in order.
struct RouterList {
  float key[68];
  int e[64];
  float sorted_key[36];
  int sorted_e[36];
};

// The groups to take from, as a mask over groups, from the values at row[0, E) in
// shared memory; false when two groups at the border are too close to tell.
// 32 / n lanes (n the next power of two) share a group and go through it from
// different places, so that groups a multiple of 32 apart use different banks.
__device__ __forceinline__ bool keep_groups(const RouterArgs& a, const float* row, bool approximate, uint32_t* keep) {
  const int lane = threadIdx.x & 31, len = a.E / a.n_group;
  const int per = a.lanes_per_group, g = lane / per, s = lane % per, turns = (len + per - 1) / per;
  float first = -INFINITY, second = -INFINITY;
  if (g < a.n_group) {
    int r = g % turns;
    for (int i = 0; i < turns; ++i) {
      const int at = s + per * r;
      const float v = at < len ? row[g * len + at] : -INFINITY;
      second = fmaxf(second, fminf(first, v));
      first = fmaxf(first, v);
      if (++r == turns) r = 0;
    }
  }
  for (int d = 1; d < per; d <<= 1) {
    const float f = __shfl_xor_sync(0xffffffffu, first, d), o = __shfl_xor_sync(0xffffffffu, second, d);
    second = fmaxf(fminf(first, f), fmaxf(second, o));
    first = fmaxf(first, f);
  }
  // off: what the score may be off, from its keys' errors (s is at most 1; the keys may be large and cancel) and the
  // sum's rounding.  An infinite key is so in truth (no expert left, or an infinite bias), and its group's score with it;
  // an infinite sum of finite keys is not.
  float score = first, off = key_error(a.sigmoid, 1.f, first);
  if (a.group_top == 2 && second != -INFINITY) {
    score += second;
    off += key_error(a.sigmoid, 1.f, second) + 1.2e-7f * fabsf(score);
  }
  const bool sure = fabsf(first) == INFINITY;
  bool tight = fabsf(score) == INFINITY && !sure && g < a.n_group;
  if (sure) off = 0.f;
  const float near = off + warp_fmax(g < a.n_group ? off : 0.f);  // with any other group's
  int before = 0;
  uint32_t close = 0;
  for (int i = 0; i < a.n_group; ++i) {
    const float o = __shfl_sync(0xffffffffu, score, i * per);
    before += o > score || (o == score && i < g);
    if (approximate && fabsf(o - score) <= near) close |= 1u << i;  // two infinities are not: NaN
  }
  const bool mine = g < a.n_group && before < a.topk_group;
  uint32_t k = __ballot_sync(0xffffffffu, mine && s == 0), m = 0;
  for (int i = 0; i < a.n_group; ++i) m |= (k >> (i * per) & 1u) << i;
  *keep = m;
  tight |= g < a.n_group && (close & (mine ? ~m : m)) != 0;
  return !__any_sync(0xffffffffu, tight);
}

// One token by one warp in fp32, NV logits a lane (all of them there if FULL): the
// K + 1 first experts in order to sorted_key and sorted_e.  False where that cannot
// be told from here (two groups too close, too many candidates): the caller then
// takes select_exact.  The K + 1 largest are among the elements that reach the
// (K + 1)-th largest of the lanes' own maxima: usually few more than K + 1, which
// are ranked against each other.  masked: there is a -inf in the row.
template <typename V, int NV, bool FULL>
__device__ __forceinline__ bool select_fast(const RouterArgs& a, const float (&x)[NV], const float (&b)[NV],
                                            const float* __restrict__ bias, bool masked, RouterList* list, float* row,
                                            float* sorted_key, int* sorted_e, float* top_logit, float* total) {
  const int lane = threadIdx.x & 31;
  const bool group_scores = a.n_group > 1 && !bias && a.group_top == 2;
  const bool scores = bias != nullptr || group_scores;
  float key[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) key[j] = x[j];
  float m = -INFINITY, z = 0.f;
  if (!a.sigmoid && (scores || !a.renorm)) {  // softmax over the row; what is not there is -inf
#pragma unroll
    for (int j = 0; j < NV; ++j) m = fmaxf(m, x[j]);
    m = warp_fmax(m);
    const float m0 = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float p = ex2_approx((x[j] - m0) * LOG2E);
      sum += p;
      key[j] = p;
    }
    z = warp_sum(sum);
  }
  *top_logit = m;
  *total = z;
  if (scores) {  // one loop to a step: a choice inside would be made for every element
    if (a.sigmoid) {
#pragma unroll
      for (int j = 0; j < NV; ++j) key[j] = rcp_approx(1.f + ex2_approx(x[j] * -LOG2E));
    } else {
      const float iz = z > 0.f ? rcp_approx(z) : 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) key[j] *= iz;
    }
    if (NV <= HOISTED) {
#pragma unroll
      for (int j = 0; j < NV; ++j) key[j] += b[j];  // 0 without a bias
    } else if (bias) {
#pragma unroll
      for (int j = 0; j < NV; ++j) key[j] += FULL || lane + 32 * j < a.E ? clean_bias(bias[lane + 32 * j]) : 0.f;
    }
    if (masked) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (x[j] == -INFINITY) key[j] = -INFINITY;
    }
  } else {
    // -0 becomes +0: they are equal, and the signs of differences below have to say so
#pragma unroll
    for (int j = 0; j < NV; ++j) key[j] = x[j] + 0.f;
  }
  // Logits that are there: not past E, nor of a group left out.  The others' keys are -inf.
  uint32_t there = 0xffffffffu;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (FULL || lane + 32 * j < a.E) row[lane + 32 * j] = key[j];
  if (a.n_group > 1) {
    uint32_t keep;
    __syncwarp();
    if (!keep_groups(a, row, scores, &keep)) return false;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (group_scores) key[j] = x[j] + 0.f;
      const uint32_t g = (uint32_t)(lane + 32 * j) * a.group_inv >> 21;
      if (!(keep >> g & 1)) {
        key[j] = -INFINITY;
        there &= ~(1u << j);
      }
    }
    if (group_scores) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (FULL || lane + 32 * j < a.E) row[lane + 32 * j] = key[j];
    }
  }
  if (!FULL) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (lane + 32 * j >= a.E) {
        key[j] = -INFINITY;
        there &= ~(1u << j);
      }
  }
  float own = NAN;
#pragma unroll
  for (int j = 0; j < NV; ++j) own = fmaxf(own, key[j]);
  float t = NAN;
  for (int k = 0; k <= a.K; k += 3) {  // up to two more than needed: t is then lower, and all that reach it are taken
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      t = warp_fmax(own);
      if (own == t) own = NAN;
    }
  }
  if (isnan(t)) t = -INFINITY;
  // Which keys reach t, by the sign of a difference (infinities of one sign give NaN, whose sign is plus): a sum and a
  // shift, where a comparison and a selection would both take the integer pipe, which is the one that is busy here.
  uint32_t below = 0;
#pragma unroll
  for (int j = NV - 1; j >= 0; --j) below = __funnelshift_l(__float_as_uint(key[j] - t), below, 1);
  uint32_t mine = ~below & there & (NV == 32 ? 0xffffffffu : (1u << NV) - 1);
  const int count = __popc(mine);
  int n = 0, at = 0;
  for (int i = 1;; ++i) {
    const uint32_t have = __ballot_sync(0xffffffffu, count >= i);
    if (!have) break;
    at += __popc(have & lanemask_lt());
    n += __popc(have);
  }
  if (n > 64) return false;
  // at: the lower lanes' candidates (those that have an i-th, summed over i), and so this lane's first place
  for (; mine; mine &= mine - 1) {
    const int e = lane + 32 * (__ffs(mine) - 1);
    list->key[at] = row[e];
    list->e[at++] = e;
  }
  if (lane < 4) list->key[n + lane] = NAN;  // the ranking goes by fours
  __syncwarp();
  const int have = min(n, a.K + 1);
  if (n <= 32 && have <= 31) {
    const float k0 = lane < n ? list->key[lane] : NAN;
    uint32_t greater = 0;  // a bit for each candidate; NaN behind them
    for (int i = 0; i < n; i += 4) {
      const float4 o = *reinterpret_cast<const float4*>(list->key + i);
      greater = __funnelshift_l(__float_as_uint(k0 - o.x), greater, 1);
      greater = __funnelshift_l(__float_as_uint(k0 - o.y), greater, 1);
      greater = __funnelshift_l(__float_as_uint(k0 - o.z), greater, 1);
      greater = __funnelshift_l(__float_as_uint(k0 - o.w), greater, 1);
    }
    const int r0 = __popc(greater);
    const bool in = lane < n && r0 < have;
    if (__reduce_or_sync(0xffffffffu, in ? 1u << r0 : 0u) == (1u << have) - 1) {  // no two of them have one rank
      if (in) {
        sorted_key[r0] = k0;
        sorted_e[r0] = list->e[lane];
      }
      return true;
    }
  }
  for (int i = lane; i < n; i += 32) {  // equal keys, or many candidates
    const float k0 = list->key[i];
    const int e0 = list->e[i];
    int r = 0;
    for (int j = 0; j < n; ++j) r += list->key[j] > k0 || (list->key[j] == k0 && list->e[j] < e0);
    if (r < have) {
      sorted_key[r] = k0;
      sorted_e[r] = e0;
    }
  }
  return true;
}

// Four consecutive elements as fp32, and back.
__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 q = *reinterpret_cast<const float4*>(p);
  v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
}
template <typename V>
__device__ __forceinline__ void load4(const V* p, float* v) {
  const uint2 q = *reinterpret_cast<const uint2*>(p);
  const V* h = reinterpret_cast<const V*>(&q);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = to_f32(h[i]);
}
__device__ __forceinline__ void store4(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <typename V>
__device__ __forceinline__ void store4(V* p, const float* v) {
  uint2 q;
  V* h = reinterpret_cast<V*>(&q);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = from_f32<V>(v[i]);
  *reinterpret_cast<uint2*>(p) = q;
}

// The end of a batch of tokens, `width` lanes to a token: lane k has its k-th
// expert id and, if `next`, that one's key and its successor's key and expert.
// Neighbours whose difference is within what both keys are off send their token to
// select_exact; then the weights.  m, z: the softmax of the lane's token.
template <typename V>
__device__ __forceinline__ void finish_tokens(const RouterArgs& a, const V* __restrict__ logits,
                                              const float* __restrict__ bias, int64_t t0, int width, bool live, int id,
                                              bool next, float key0, float key1, int e1, float m, float z,
                                              double* exact_keys, int32_t* __restrict__ ids, float* __restrict__ w) {
  const int lane = threadIdx.x & 31, of = lane / width, k = lane % width;
  const V* row = logits + (t0 + of) * a.ld;
  if (bias) {
    bool tight = false;
    // A score of 1 bounds every error.  Between two chosen ones the errors of their own scores decide where that is not
    // enough (one that overtakes several lies within them of the one before it); behind the last one stand experts whose
    // keys are not at hand, so there any score has to be allowed for.  With a softmax that is wide against keys of about
    // 1 / E: 524,288 tokens over 384 experts, K = 8, take 507 us where logits spread by 1 (284 without a bias) and 961 where
    // they spread by 0.3; 262,144 over 1024 experts 870 and 2260 (278).
    tight = next && key1 != -INFINITY && key0 != INFINITY &&  // infinite keys are so in truth
            key0 - key1 <= key_error(a.sigmoid, 1.f, key0) + key_error(a.sigmoid, 1.f, key1);
    if (tight && k + 1 < a.K) {
      const float b0 = bias[id], b1 = bias[e1];
      tight = key0 - key1 <= key_error(a.sigmoid, key0 - b0, key0) + key_error(a.sigmoid, key1 - b1, key1);
      if (tight && b0 == b1) tight = to_f32(row[id]) != to_f32(row[e1]);  // equal in truth: in order as it is
    }
    uint32_t again = __ballot_sync(0xffffffffu, tight);
    while (again) {
      const int i = (__ffs(again) - 1) / width;
      const int e = select_exact(a, logits + (t0 + i) * a.ld, bias, exact_keys);
      const int back = __shfl_sync(0xffffffffu, e, k);
      if (of == i && live) id = back;
      again &= ~((width == 32 ? 0xffffffffu : (1u << width) - 1) << (i * width));
      __syncwarp();
    }
  }
  bool ignore = false;
  const float x = live ? clean_logit(to_f32(row[id]), ignore) : -INFINITY;
  float v;
  if (a.renorm)
    v = chosen_ratio(x, a.sigmoid, width);
  else if (a.sigmoid)
    v = sigmoid_f32(x);
  else
    v = m == -INFINITY ? 0.f : exp_near(x - m) / z;
  if (live) {
    const int64_t to = (t0 + of) * a.K + k;
    ids[to] = id;
    w[to] = a.scale * v;
  }
}

// A warp takes 32 / width tokens at a time: one after the other as far as the
// choice goes, then together, width lanes a token (the next power of two from K,
// at least 8), for what concerns the K chosen ones only.  A warp to a token the
// whole way took 420 us where this took 365 (524,288 tokens, 384 experts).
template <typename V, int NV, bool FULL>
__global__ void __launch_bounds__(ROUTER_WARPS * 32, NV <= 12 ? 4 : NV <= 16 ? 3 : 2)
    k_router(const V* __restrict__ logits, const float* __restrict__ bias, RouterArgs a, int32_t* __restrict__ ids,
             float* __restrict__ w, int32_t* dev_status) {
  extern __shared__ double s_key[];  // [warps][E], of select_exact (select_fast uses it as fp32)
  __shared__ __align__(16) RouterList s_list[ROUTER_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double* mine = s_key + (size_t)warp * a.E;
  RouterList* list = s_list + warp;
  const int width = a.width, batch = 32 / width, of = lane / width, k = lane % width;
  wait_for_predecessor();
  float b[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j)
    b[j] = NV <= HOISTED && bias && (FULL || lane + 32 * j < a.E) ? clean_bias(bias[lane + 32 * j]) : 0.f;
  const int64_t t0 = ((int64_t)blockIdx.x * ROUTER_WARPS + warp) * batch;
  if (t0 < a.T) {
    const int n = (int)min((int64_t)batch, a.T - t0);
    float m = 0.f, z = 0.f;     // softmax of this lane's token
    uint32_t exact = 0;         // tokens whose choice is from select_exact
    for (int i = 0; i < n; ++i) {
      const V* row = logits + (t0 + i) * a.ld;
      float x[NV];
      bool special = false;
#pragma unroll
      for (int j = 0; j < NV; ++j) x[j] = FULL || lane + 32 * j < a.E ? to_f32(row[lane + 32 * j]) : -INFINITY;
      if (FULL) {  // an infinity or NaN times 0 is NaN
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) sum = fmaf(x[j], 0.f, sum);
        special = sum != 0.f;
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) special |= !(fabsf(x[j]) <= FLT_MAX) && lane + 32 * j < a.E;
      }
      special = __any_sync(0xffffffffu, special);
      if (special) {
        bool bad = false;
#pragma unroll
        for (int j = 0; j < NV; ++j) x[j] = clean_logit(x[j], bad);
        if (__any_sync(0xffffffffu, bad) && lane == 0) flag(dev_status, EP_DEV_BAD_LOGIT);
      }
      float mi, zi;
      int* to = list->sorted_e + i * (a.K + 1);
      if (!select_fast<V, NV, FULL>(a, x, b, bias, special, list, reinterpret_cast<float*>(mine),
                                    list->sorted_key + i * (a.K + 1), to, &mi, &zi)) {
        __syncwarp();
        const int id = select_exact(a, row, bias, mine);
        if (lane < a.K) to[lane] = id;
        exact |= 1u << i;
      }
      if (of == i) {
        m = mi;
        z = zi;
      }
      __syncwarp();
    }
    const int at = of * (a.K + 1) + k;
    const bool live = of < n && k < a.K;
    // the (K + 1)-th is there unless there are only K
    const bool next = live && !(exact >> of & 1) && (k + 1 < a.K || a.more);
    finish_tokens(a, logits, bias, t0, width, live, live ? list->sorted_e[at] : 0, next,
                  next ? list->sorted_key[at] : 0.f, next ? list->sorted_key[at + 1] : 0.f,
                  next ? list->sorted_e[at + 1] : 0, m, z, mine, ids, w);
  }
}

// Many tokens over few experts (up to 8 * NE = 128, no groups, K up to 8): eight
// lanes to a token, four tokens at once.  Each round takes the largest key over the
// eight lanes, the lowest index where several have it, and strikes it out: what a
// round costs is shared by four tokens, where a warp to a token spends it on one.
// (262,144 tokens over 64 experts, softmax, K = 6: 58 us against 120; over 128
// experts, K = 8: 99 against 118.)  Lane l has the elements 32 i + 4 l + j.
template <typename V, int NE, bool VEC>
__global__ void __launch_bounds__(ROUTER_WARPS * 32)
    k_router_small(const V* __restrict__ logits, const float* __restrict__ bias, RouterArgs a,
                   int32_t* __restrict__ ids, float* __restrict__ w, int32_t* dev_status) {
  extern __shared__ double s_key[];  // [warps][E], of select_exact
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, of = lane >> 3, l = lane & 7;
  wait_for_predecessor();
  const int64_t t0 = ((int64_t)blockIdx.x * ROUTER_WARPS + warp) * 4;
  if (t0 >= a.T) return;
  const int n = (int)min((int64_t)4, a.T - t0);
  const V* row = logits + (t0 + min(of, n - 1)) * a.ld;  // lanes without a token repeat the last one's
  float x[NE], key[NE];
#pragma unroll
  for (int i = 0; i < NE / 4; ++i) {
    const int e = 32 * i + 4 * l;
    if (VEC) {
      if (e < a.E) {
        load4(row + e, x + 4 * i);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * i + j] = -INFINITY;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[4 * i + j] = e + j < a.E ? to_f32(row[e + j]) : -INFINITY;
    }
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NE; ++i) bad |= !(x[i] <= FLT_MAX);
  if (__any_sync(0xffffffffu, bad)) {
#pragma unroll
    for (int i = 0; i < NE; ++i) x[i] = clean_logit(x[i], bad);
    if (lane == 0) flag(dev_status, EP_DEV_BAD_LOGIT);
  }
  float m = -INFINITY, z = 0.f;
#pragma unroll
  for (int i = 0; i < NE; ++i) key[i] = x[i];
  if (!a.sigmoid && (bias || !a.renorm)) {  // softmax over the row
#pragma unroll
    for (int i = 0; i < NE; ++i) m = fmaxf(m, x[i]);
#pragma unroll
    for (int d = 4; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float m0 = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const float p = ex2_approx((x[i] - m0) * LOG2E);
      z += p;
      if (bias) key[i] = p;
    }
#pragma unroll
    for (int d = 4; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
  }
  if (bias) {
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < NE; ++i) key[i] = rcp_approx(1.f + ex2_approx(x[i] * -LOG2E));
    } else {
      const float iz = z > 0.f ? rcp_approx(z) : 0.f;
#pragma unroll
      for (int i = 0; i < NE; ++i) key[i] *= iz;
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = 32 * (i / 4) + 4 * l + i % 4;
      key[i] += e < a.E ? clean_bias(bias[e]) : 0.f;
      if (x[i] == -INFINITY) key[i] = -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < NE; ++i)
    if (32 * (i / 4) + 4 * l + i % 4 >= a.E) key[i] = NAN;  // not there
  // lane k of a token keeps its k-th expert; the (K + 1)-th, for the one before it, every lane does
  const int rounds = a.K + (bias && a.more ? 1 : 0);
  float mine = 0.f, last = 0.f;
  int id = 0, last_e = 0;
  for (int r = 0; r < rounds; ++r) {
    float g = NAN;
#pragma unroll
    for (int i = 0; i < NE; ++i) g = fmaxf(g, key[i]);
#pragma unroll
    for (int d = 4; d; d >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, d));
    int at = NE;
#pragma unroll
    for (int i = NE - 1; i >= 0; --i) at = key[i] == g ? i : at;
    const int e = at < NE ? 32 * (at >> 2) + 4 * l + (at & 3) : INT_MAX;
    int first = e;
#pragma unroll
    for (int d = 4; d; d >>= 1) first = min(first, __shfl_xor_sync(0xffffffffu, first, d));
    if (first != e) at = NE;
#pragma unroll
    for (int i = 0; i < NE; ++i) key[i] = i == at ? NAN : key[i];
    if (l == r) {
      mine = g;
      id = first;
    }
    last = g;
    last_e = first;
  }
  const bool live = of < n && l < a.K;
  const float after = __shfl_down_sync(0xffffffffu, mine, 1);
  const int after_e = __shfl_down_sync(0xffffffffu, id, 1);
  finish_tokens(a, logits, bias, t0, 8, live, live ? id : 0, live && (l + 1 < a.K || a.more), mine,
                l + 1 < a.K ? after : last, l + 1 < a.K ? after_e : last_e, m, z, s_key + (size_t)warp * a.E, ids, w);
}

// The gradient of the weights.  With r_k = s_k / sum_j s_j:
//   softmax, renorm   dx_k = scale r_k (dw_k - i),            i = sum_j dw_j r_j
//   sigmoid, renorm   dx_k = scale r_k (1 - s_k) (dw_k - i)
//   sigmoid           dx_k = scale s_k (1 - s_k) dw_k
//   softmax           dx_e = scale s_e ([e chosen] dw_e - i), i = sum_j dw_j s_j
// Only the last touches experts that were not chosen (and has to read the row).
// An expert that stands twice among a token's ids gets the sum of its terms.
//
// Bound by writing dlogits.  As in the router, a warp takes 32 / width tokens: the
// chosen logits of all of them at once, then row by row.  The chosen experts'
// terms are laid into a row of zeros in shared memory, the row goes out in vectors
// of four (VEC: the rows are aligned to that), and only the places that were
// written are zeroed again.
template <typename V, int NC, bool VEC>
__global__ void __launch_bounds__(ROUTER_WARPS * 32)
    k_router_backward(const float* __restrict__ dw, const V* __restrict__ logits, const int32_t* __restrict__ ids,
                      RouterArgs a, int64_t ld_out, V* __restrict__ dlogits, int32_t* dev_status) {
  extern __shared__ __align__(16) float s_row[];  // [warps][NC * 128]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* out = s_row + warp * (NC * 128);
  const int width = a.width, batch = 32 / width, of = lane / width, k = lane % width;
  const bool dense = !a.sigmoid && !a.renorm;
#pragma unroll
  for (int c = 0; c < NC; ++c) *reinterpret_cast<float4*>(out + c * 128 + lane * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncwarp();
  wait_for_predecessor();
  uint32_t bits = 0;
  const int64_t t0 = ((int64_t)blockIdx.x * ROUTER_WARPS + warp) * batch;
  if (t0 < a.T) {
    const int n = (int)min((int64_t)batch, a.T - t0);
    bool bad = false;
    int id = -1;
    float x = -INFINITY, d = 0.f;
    if (of < n && k < a.K) {
      const int64_t at = (t0 + of) * a.K + k;
      id = ids[at];
      if (id < 0 || id >= a.E) {
        bits |= EP_DEV_BAD_EXPERT_ID;
        id = -1;
      } else {
        d = dw[at];
        x = clean_logit(to_f32(logits[(t0 + of) * a.ld + id]), bad);
      }
    }
    float v = 0.f;  // this lane's term of dlogits[id], without the scale
    if (a.renorm) {
      const float r = chosen_ratio(x, a.sigmoid, width);
      float i = d * r;
      for (int s = width >> 1; s; s >>= 1) i += __shfl_xor_sync(0xffffffffu, i, s);
      v = r * (d - i);
      if (a.sigmoid) v *= sigmoid_f32(-x);
    } else if (a.sigmoid) {
      v = d * sigmoid_f32(x) * sigmoid_f32(-x);
    }
    // of lanes with the same expert of the same token, the first lays down the sum of all, in order
    uint32_t same = 0;
    for (int j = 0; j < a.K; ++j) same |= __shfl_sync(0xffffffffu, id, of * width + j) == id ? 1u << j : 0u;
    const bool lead = id >= 0 && (same & ((1u << k) - 1)) == 0;
    const bool twice = __any_sync(0xffffffffu, id >= 0 && (same & (same - 1)));
    for (int i = 0; i < n; ++i) {
      const V* row = logits + (t0 + i) * a.ld;
      V* to = dlogits + (t0 + i) * ld_out;
      float p[NC][4], inner = 0.f;
      if (dense) {
        float m = -INFINITY, z = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
#pragma unroll
          for (int j = 0; j < 4; ++j) p[c][j] = -INFINITY;
          const int e = c * 128 + lane * 4;
          if (VEC) {
            if (e < a.E) load4(row + e, p[c]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (e + j < a.E) p[c][j] = to_f32(row[e + j]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            p[c][j] = clean_logit(p[c][j], bad);
            m = fmaxf(m, p[c][j]);
          }
        }
        m = warp_fmax(m);
        const float m0 = m == -INFINITY ? 0.f : m;  // a row of -inf has scores of 0
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) z += p[c][j] = exp_near(p[c][j] - m0);
        z = warp_sum(z);
        const float iz = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) p[c][j] *= iz;
        float s = of == i ? d * (exp_near(x - m0) * iz) : 0.f;
        if (of == i) v = s;
        inner = warp_sum(s) * a.scale;
      }
      float mine = a.scale * v;
      if (twice) {
        float sum = 0.f;
        for (int j = 0; j < a.K; ++j) {
          const float o = __shfl_sync(0xffffffffu, mine, of * width + j);
          if (same >> j & 1) sum += o;
        }
        mine = sum;
      }
      if (lead && of == i) out[id] = mine;
      __syncwarp();
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int e = c * 128 + lane * 4;
        if (e < a.E) {
          const float4 q = *reinterpret_cast<const float4*>(out + e);
          float o[4] = {q.x, q.y, q.z, q.w};
          if (dense) {
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] -= inner * p[c][j];
          }
          if (VEC) {
            store4(to + e, o);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (e + j < a.E) to[e + j] = from_f32<V>(o[j]);
          }
        }
      }
      __syncwarp();
      if (lead && of == i) out[id] = 0.f;
    }
    if (bad) bits |= EP_DEV_BAD_LOGIT;
  }
  bits = __reduce_or_sync(0xffffffffu, bits);
  if (bits && lane == 0) flag(dev_status, bits);
}

// The same for many tokens over few experts: eight lanes to a token as in
// k_router_small, four tokens at once.  (262,144 tokens over 64 experts, softmax over
// all, K = 6, bf16: 33 us against 82.)
template <typename V, int NE, bool VEC>
__global__ void __launch_bounds__(ROUTER_WARPS * 32)
    k_router_backward_small(const float* __restrict__ dw, const V* __restrict__ logits,
                            const int32_t* __restrict__ ids, RouterArgs a, int64_t ld_out, V* __restrict__ dlogits,
                            int32_t* dev_status) {
  __shared__ __align__(16) float s_row[ROUTER_WARPS * 4 * 8 * NE];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, of = lane >> 3, l = lane & 7;
  float* out = s_row + (warp * 4 + of) * 8 * NE;  // this token's row
#pragma unroll
  for (int i = 0; i < NE / 4; ++i) *reinterpret_cast<float4*>(out + 32 * i + 4 * l) = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncwarp();
  wait_for_predecessor();
  const int64_t t0 = ((int64_t)blockIdx.x * ROUTER_WARPS + warp) * 4;
  if (t0 >= a.T) return;
  const int n = (int)min((int64_t)4, a.T - t0);
  const int64_t t = t0 + min(of, n - 1);
  const V* row = logits + t * a.ld;
  const bool dense = !a.sigmoid && !a.renorm, live = of < n && l < a.K;
  uint32_t bits = 0;
  bool bad = false;
  int id = -1;
  float x = -INFINITY, d = 0.f;
  if (live) {
    id = ids[t * a.K + l];
    if (id < 0 || id >= a.E) {
      bits |= EP_DEV_BAD_EXPERT_ID;
      id = -1;
    } else {
      d = dw[t * a.K + l];
      x = clean_logit(to_f32(row[id]), bad);
    }
  }
  float p[NE], v = 0.f, inner = 0.f;  // v: this lane's term of dlogits[id], without the scale
  if (dense) {
    float m = -INFINITY, z = 0.f;
#pragma unroll
    for (int i = 0; i < NE / 4; ++i) {
      const int e = 32 * i + 4 * l;
#pragma unroll
      for (int j = 0; j < 4; ++j) p[4 * i + j] = -INFINITY;
      if (VEC) {
        if (e < a.E) load4(row + e, p + 4 * i);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (e + j < a.E) p[4 * i + j] = to_f32(row[e + j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[4 * i + j] = clean_logit(p[4 * i + j], bad);
        m = fmaxf(m, p[4 * i + j]);
      }
    }
#pragma unroll
    for (int s = 4; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
    const float m0 = m == -INFINITY ? 0.f : m;  // a row of -inf has scores of 0
#pragma unroll
    for (int i = 0; i < NE; ++i) z += p[i] = exp_near(p[i] - m0);
#pragma unroll
    for (int s = 4; s; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
    const float iz = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) p[i] *= iz;
    v = d * (exp_near(x - m0) * iz);
    inner = v;
#pragma unroll
    for (int s = 4; s; s >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, s);
    inner *= a.scale;
  } else if (a.renorm) {
    const float r = chosen_ratio(x, a.sigmoid, 8);
    float i = d * r;
#pragma unroll
    for (int s = 4; s; s >>= 1) i += __shfl_xor_sync(0xffffffffu, i, s);
    v = r * (d - i);
    if (a.sigmoid) v *= sigmoid_f32(-x);
  } else {
    v = d * sigmoid_f32(x) * sigmoid_f32(-x);
  }
  // of lanes with the same expert of the same token, the first lays down the sum of all, in order
  float mine = a.scale * v;
  uint32_t same = 0;
  for (int j = 0; j < a.K; ++j) same |= __shfl_sync(0xffffffffu, id, of * 8 + j) == id ? 1u << j : 0u;
  if (__any_sync(0xffffffffu, id >= 0 && (same & (same - 1)))) {
    float sum = 0.f;
    for (int j = 0; j < a.K; ++j) {
      const float o = __shfl_sync(0xffffffffu, mine, of * 8 + j);
      if (same >> j & 1) sum += o;
    }
    mine = sum;
  }
  if (id >= 0 && (same & ((1u << l) - 1)) == 0) out[id] = mine;
  __syncwarp();
  V* to = dlogits + t * ld_out;
#pragma unroll
  for (int i = 0; i < NE / 4; ++i) {
    const int e = 32 * i + 4 * l;
    if (of < n && e < a.E) {
      const float4 q = *reinterpret_cast<const float4*>(out + e);
      float o[4] = {q.x, q.y, q.z, q.w};
      if (dense) {
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] -= inner * p[4 * i + j];
      }
      if (VEC) {
        store4(to + e, o);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (e + j < a.E) to[e + j] = from_f32<V>(o[j]);
      }
    }
  }
  if (bad) bits |= EP_DEV_BAD_LOGIT;
  bits = __reduce_or_sync(0xffffffffu, bits);
  if (bits && lane == 0) flag(dev_status, bits);
}

static bool valid_router(int dtype, int64_t T, int E, int64_t ld, int K, int score, float scale) {
  if (!valid_tke(T, K, E) || ld < E) return false;
  if (dtype != EP_DTYPE_F32 && dtype != EP_DTYPE_BF16 && dtype != EP_DTYPE_F16) return false;
  return (score == EP_SCORE_SOFTMAX || score == EP_SCORE_SIGMOID) && isfinite(scale);
}

static bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Few tokens: one to a warp, they are all at work at once.
static int router_width(const RouterArgs& a) {
  return a.T <= (int64_t)num_sms() * 32 ? 32 : a.K <= 8 ? 8 : a.K <= 16 ? 16 : 32;
}

template <typename V, int NV, bool FULL>
static int launch_router(const void* logits, const float* bias, const RouterArgs& a, int32_t* ids, float* w,
                         int32_t* dev_status, cudaStream_t stream) {
  const size_t smem = (size_t)ROUTER_WARPS * a.E * sizeof(double);
  if (!raise_smem_limit((const void*)k_router<V, NV, FULL>, smem)) return EP_ERR_CUDA;
  // one batch a warp, not a resident grid that goes on to the next: 356 against 366 us, with groups 292 against 323
  const int64_t per = ROUTER_WARPS * (32 / a.width);
  void* args[] = {&logits, &bias, (void*)&a, &ids, &w, &dev_status};
  if (launch_pdl((const void*)k_router<V, NV, FULL>, dim3((unsigned)((a.T + per - 1) / per)), dim3(ROUTER_WARPS * 32),
                 args, smem, stream) != cudaSuccess)
    return EP_ERR_CUDA;
  count_launch();
  return EP_OK;
}

template <typename V, int NE>
static int launch_small(const void* logits, const float* bias, const RouterArgs& a, int32_t* ids, float* w,
                        int32_t* dev_status, cudaStream_t stream) {
  const bool vec = a.E % 4 == 0 && a.ld % 4 == 0 && aligned_to(logits, 4 * sizeof(V));
  const void* fn = vec ? (const void*)k_router_small<V, NE, true> : (const void*)k_router_small<V, NE, false>;
  void* args[] = {&logits, &bias, (void*)&a, &ids, &w, &dev_status};
  if (launch_pdl(fn, dim3((unsigned)((a.T + 4 * ROUTER_WARPS - 1) / (4 * ROUTER_WARPS))), dim3(ROUTER_WARPS * 32), args,
                 (size_t)ROUTER_WARPS * a.E * sizeof(double), stream) != cudaSuccess)
    return EP_ERR_CUDA;
  count_launch();
  return EP_OK;
}

template <typename V>
static int run_router(const void* logits, const float* bias, RouterArgs a, int32_t* ids, float* w, int32_t* dev_status,
                      cudaStream_t stream) {
  a.lanes_per_group = 32;
  while (a.lanes_per_group * a.n_group > 32) a.lanes_per_group /= 2;
  const int len = a.E / a.n_group;
  a.more = (a.n_group == 1 ? a.E : a.topk_group * len) > a.K;
  a.width = router_width(a);
  a.group_inv = ((1u << 21) + len - 1) / len;
  if (a.width == 8 && a.n_group == 1 && a.E <= SMALL_E) {
    if (a.E <= 64) return launch_small<V, 8>(logits, bias, a, ids, w, dev_status, stream);
    return launch_small<V, 16>(logits, bias, a, ids, w, dev_status, stream);
  }
  // logits a lane: the next of these up from E / 32
#define EP_ROUTER(nv)                                                                       \
  if (a.E == 32 * nv) return launch_router<V, nv, true>(logits, bias, a, ids, w, dev_status, stream); \
  if (a.E < 32 * nv) return launch_router<V, nv, false>(logits, bias, a, ids, w, dev_status, stream)
  EP_ROUTER(2);
  EP_ROUTER(4);
  EP_ROUTER(8);
  EP_ROUTER(12);
  EP_ROUTER(16);
  EP_ROUTER(32);
#undef EP_ROUTER
  return EP_ERR_ARG;
}

template <typename V, int NC, bool VEC>
static int launch_backward(const float* dw, const void* logits, const int32_t* ids, const RouterArgs& a, int64_t ld_out,
                           void* dlogits, int32_t* dev_status, cudaStream_t stream) {
  const size_t smem = (size_t)ROUTER_WARPS * NC * 128 * sizeof(float);
  if (!raise_smem_limit((const void*)k_router_backward<V, NC, VEC>, smem)) return EP_ERR_CUDA;
  // one batch a warp: 188 us against 219 with a resident grid (524,288 tokens, 384 experts)
  const int64_t per = ROUTER_WARPS * (32 / a.width);
  void* args[] = {&dw, &logits, &ids, (void*)&a, &ld_out, &dlogits, &dev_status};
  if (launch_pdl((const void*)k_router_backward<V, NC, VEC>, dim3((unsigned)((a.T + per - 1) / per)),
                 dim3(ROUTER_WARPS * 32), args, smem, stream) != cudaSuccess)
    return EP_ERR_CUDA;
  count_launch();
  return EP_OK;
}

template <typename V>
static int run_router_backward(const float* dw, const void* logits, const int32_t* ids, RouterArgs a, int64_t ld_out,
                               void* dlogits, int32_t* dev_status, cudaStream_t stream) {
  a.width = router_width(a);
  const bool vec = a.E % 4 == 0 && a.ld % 4 == 0 && ld_out % 4 == 0 && aligned_to(logits, 4 * sizeof(V)) &&
                   aligned_to(dlogits, 4 * sizeof(V));
  if (a.width == 8 && a.E <= SMALL_E) {
    const void* fn = a.E <= 64 ? vec ? (const void*)k_router_backward_small<V, 8, true>
                                     : (const void*)k_router_backward_small<V, 8, false>
                               : vec ? (const void*)k_router_backward_small<V, 16, true>
                                     : (const void*)k_router_backward_small<V, 16, false>;
    void* args[] = {&dw, &logits, &ids, (void*)&a, &ld_out, &dlogits, &dev_status};
    if (launch_pdl(fn, dim3((unsigned)((a.T + 4 * ROUTER_WARPS - 1) / (4 * ROUTER_WARPS))), dim3(ROUTER_WARPS * 32),
                   args, 0, stream) != cudaSuccess)
      return EP_ERR_CUDA;
    count_launch();
    return EP_OK;
  }
#define EP_BACKWARD(nc)                                                                                            \
  if (a.E <= 128 * nc)                                                                                             \
  return vec ? launch_backward<V, nc, true>(dw, logits, ids, a, ld_out, dlogits, dev_status, stream)               \
             : launch_backward<V, nc, false>(dw, logits, ids, a, ld_out, dlogits, dev_status, stream)
  EP_BACKWARD(1);
  EP_BACKWARD(2);
  EP_BACKWARD(4);
  EP_BACKWARD(8);
#undef EP_BACKWARD
  return EP_ERR_ARG;
}

}  // namespace ep

using namespace ep;

extern "C" int ep_router(const void* logits, int dtype, int64_t T, int E, int64_t ld, int K, int score,
                         const float* bias, int n_group, int topk_group, int group_top, int renorm, float scale,
                         int32_t* topk_ids, float* w, int32_t* dev_status, cudaStream_t stream) {
  if (!valid_router(dtype, T, E, ld, K, score, scale)) return EP_ERR_ARG;
  if (n_group < 1 || n_group > 32 || E % n_group || topk_group < 1 || topk_group > n_group ||
      (int64_t)topk_group * (E / n_group) < K || (group_top != 1 && group_top != 2))
    return EP_ERR_ARG;
  if (T == 0) return EP_OK;
  if (!logits || !topk_ids || !w || !aligned_to(logits, dtype == EP_DTYPE_F32 ? 4 : 2) || !aligned_to(bias, 4) ||
      !aligned_to(topk_ids, 4) || !aligned_to(w, 4))
    return EP_ERR_ARG;
  const RouterArgs a{T, ld, E, K, topk_group == n_group ? 1 : n_group, topk_group, group_top,
                     score == EP_SCORE_SIGMOID, renorm != 0, scale, 32, true, 32, 0};
  if (dtype == EP_DTYPE_F32) return run_router<float>(logits, bias, a, topk_ids, w, dev_status, stream);
  if (dtype == EP_DTYPE_BF16) return run_router<__nv_bfloat16>(logits, bias, a, topk_ids, w, dev_status, stream);
  return run_router<__half>(logits, bias, a, topk_ids, w, dev_status, stream);
}

extern "C" int ep_router_backward(const float* dw, const void* logits, int dtype, int64_t T, int E, int64_t ld,
                                  const int32_t* topk_ids, int K, int score, int renorm, float scale, void* dlogits,
                                  int64_t ld_out, int32_t* dev_status, cudaStream_t stream) {
  if (!valid_router(dtype, T, E, ld, K, score, scale) || ld_out < E) return EP_ERR_ARG;
  if (T == 0) return EP_OK;
  const size_t size = dtype == EP_DTYPE_F32 ? 4 : 2;
  if (!dw || !logits || !topk_ids || !dlogits || !aligned_to(logits, size) || !aligned_to(dlogits, size) ||
      !aligned_to(dw, 4) || !aligned_to(topk_ids, 4))
    return EP_ERR_ARG;
  const RouterArgs a{T, ld, E, K, 1, 1, 1, score == EP_SCORE_SIGMOID, renorm != 0, scale, 32, true, 32, 0};
  if (dtype == EP_DTYPE_F32)
    return run_router_backward<float>(dw, logits, topk_ids, a, ld_out, dlogits, dev_status, stream);
  if (dtype == EP_DTYPE_BF16)
    return run_router_backward<__nv_bfloat16>(dw, logits, topk_ids, a, ld_out, dlogits, dev_status, stream);
  return run_router_backward<__half>(dw, logits, topk_ids, a, ld_out, dlogits, dev_status, stream);
}
