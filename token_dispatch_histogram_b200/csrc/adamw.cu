// One AdamW step over many tensors at once, behind the replica gradient
// reduction: element by element, with g the gradient (scaled), t the step,
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - (m lr / (1 - b1^t)) / (sqrt(v) / sqrt(1 - b2^t) + eps)
// and optionally the bf16 copy of p that the experts' products read.
//
// The moments are fp32, or 8 bits in blocks of 256 elements with one fp32 scale
// each: e4m3 codes, the block's largest magnitude at 448.  The second moment is
// held as its root (its range is that of |g| then), and a nonzero root never at
// code 0, which a later step would divide by.  A step computes with the moments
// before they are coded again.
//
// A step moves v by the share c = (1 - b2) / (1 - b2^t) of g^2 - v at most.  A
// code is 6 to 12 % of a root: rounded to nearest, roots stand still once c is so
// small that hardly a step moves one by half of that (b2 = 0.999, half of the
// gradients changed fivefold: 3000 steps later their roots were a third, or three
// times, of fp32's).  From c < 1/32 on, roots that had a value are therefore
// rounded up or down by chance, in proportion, so that they follow v on average
// (0.99 to 1.02 of fp32's there, 15 to 25 % around it).  The chance is a hash of
// step and element: the same step gives the same codes.  The first moment's share
// is 1 - b1 of a gradient that is mostly noise, which moves its codes; it is
// rounded to nearest.
//
// Every product, sum, quotient and root is rounded by itself, in the order
// above, so the codes do not depend on how a compiler joins operations.
//
// Bound by memory: 28 bytes an element with fp32 moments, 16 with 8 bits, 2 more
// for the copy.  A block of 256 elements belongs to one warp, eight consecutive
// elements to a lane, so a lane's codes are 8 bytes and a block's maximum is a
// shuffle reduction; nothing is shared between warps.
#include <cuda_fp8.h>
#include <math.h>

#include "common.cuh"

namespace ep {

constexpr int ADAM_BLOCK = EP_ADAMW_BLOCK;
constexpr int ADAM_WARPS = 8;
constexpr int ADAM_TENSORS = 256;  // of one launch: the table is a kernel parameter
constexpr int ADAM_FEW = 16;       // up to so many go as a parameter of 1.2 KB instead of 19: 0.9 us less to launch
constexpr float FP8_MAX = 448.f, FP8_MIN = 0x1p-9f, FP8_TINY = 0x1p-100f;

template <int CAP>
struct AdamTable {
  EpAdamWTensor t[CAP];
  int32_t before[CAP + 1];  // blocks of 256 elements before each tensor
  int n;
};

struct AdamArgs {
  double lr, b1, b2, eps, wd;
  const float* lr_dev;
  const float* grad_scale;
  const int32_t* step;
};

// What the elements need of the step, in fp32: computed once per CTA in fp64.
struct AdamConst {
  float b1, b2, c1m, c2m, decay, c1, c2, eps, gs;
  uint32_t chance;  // 8 bits: a seed of this step's roundings, or 0: to nearest
};

constexpr double NEAREST_SHARE = 1.0 / 32;  // of g^2 in v, down to which roots are rounded to nearest

// A bijection of 32 bits that spreads each bit over all (xorshift and multiply steps).
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7feb352du;
  x ^= x >> 15;
  x *= 0x846ca68bu;
  return x ^ x >> 16;
}

__device__ __forceinline__ AdamConst adam_const(const AdamArgs& a) {
  const double t = *a.step, lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
  AdamConst c;
  c.b1 = (float)a.b1;
  c.b2 = (float)a.b2;
  c.c1m = (float)(1.0 - a.b1);
  c.c2m = (float)(1.0 - a.b2);
  c.decay = (float)(1.0 - lr * a.wd);
  c.c1 = (float)(lr / (1.0 - pow(a.b1, t)));
  const double part = 1.0 - pow(a.b2, t);
  c.c2 = (float)(1.0 / sqrt(part));
  c.chance = 1.0 - a.b2 < NEAREST_SHARE * part ? mix32((uint32_t)*a.step) | 1u : 0u;
  c.eps = (float)a.eps;
  c.gs = a.grad_scale ? *a.grad_scale : 1.f;
  return c;
}

__device__ __forceinline__ void adam_element(const AdamConst& c, bool scaled, float& p, float g, float& m, float& v,
                                             float& root) {
  if (scaled) g = __fmul_rn(g, c.gs);
  m = __fadd_rn(__fmul_rn(m, c.b1), __fmul_rn(g, c.c1m));
  v = __fadd_rn(__fmul_rn(v, c.b2), __fmul_rn(__fmul_rn(g, g), c.c2m));
  root = __fsqrt_rn(v);
  p = __fsub_rn(__fmul_rn(p, c.decay),
                __fdiv_rn(__fmul_rn(m, c.c1), __fadd_rn(__fmul_rn(root, c.c2), c.eps)));
}

// Eight consecutive elements from i on, those below n; whole and aligned ones as two 16-byte accesses.
__device__ __forceinline__ void load8(const float* p, int64_t i, int64_t n, bool vec, float* x) {
  if (vec && i + 8 <= n) {
    const float4 a = *reinterpret_cast<const float4*>(p + i), b = *reinterpret_cast<const float4*>(p + i + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = i + j < n ? p[i + j] : 0.f;
  }
}

__device__ __forceinline__ void store8(float* p, int64_t i, int64_t n, bool vec, const float* x) {
  if (vec && i + 8 <= n) {
    *reinterpret_cast<float4*>(p + i) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + i + 4) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) p[i + j] = x[j];
  }
}

__device__ __forceinline__ void load8_bf16(const uint16_t* p, int64_t i, int64_t n, bool vec, float* x) {
  if (vec && i + 8 <= n) {
    const uint4 q = *reinterpret_cast<const uint4*>(p + i);
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = bf16_bits_to_f32(u[j] & 0xffffu);
      x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = i + j < n ? bf16_bits_to_f32(p[i + j]) : 0.f;
  }
}

__device__ __forceinline__ void store8_bf16(uint16_t* p, int64_t i, int64_t n, bool vec, const float* x) {
  const uint32_t u[4] = {f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]), f32x2_to_bf16x2(x[4], x[5]),
                         f32x2_to_bf16x2(x[6], x[7])};
  if (vec && i + 8 <= n) {
    *reinterpret_cast<uint4*>(p + i) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) p[i + j] = (uint16_t)(u[j >> 1] >> (j & 1) * 16);
  }
}

__device__ __forceinline__ void load8_codes(const uint8_t* p, int64_t i, int64_t n, bool vec, float scale, float* x) {
  uint32_t w[2] = {0, 0};
  if (vec && i + 8 <= n) {
    const uint2 q = *reinterpret_cast<const uint2*>(p + i);
    w[0] = q.x, w[1] = q.y;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) w[j >> 2] |= (uint32_t)p[i + j] << (j & 3) * 8;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // two codes to two halves, exactly
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j >> 1] >> (j & 1) * 16), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x[2 * j] = __fmul_rn(f.x, scale);
    x[2 * j + 1] = __fmul_rn(f.y, scale);
  }
}

// A positive value below 480 to one of its two neighbours among the codes' values, `bits` (20 of them) being the chance:
// added below the last place that a code holds, then cut off there.  Below 2^-6 the codes are multiples of 2^-9.
__device__ __forceinline__ float round_by_chance(float y, uint32_t bits) {
  if (y < 0x1p-6f) return floorf(fmaf(y, 0x1p9f, (float)bits * 0x1p-20f)) * 0x1p-9f;
  return __uint_as_float((__float_as_uint(y) + bits) & 0xfff00000u);
}

// Codes of a block's eight values a lane, and the block's scale (the same on every lane).  CHANCE: those of the eight
// that `had` a value before are rounded by the lane's chance, otherwise to nearest.
template <bool ROOT, bool CHANCE>
__device__ __forceinline__ float store8_codes(uint8_t* p, int64_t i, int64_t n, bool vec, const float* x,
                                              uint32_t chance, uint32_t had) {
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));  // a NaN keeps to its own element
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  const bool held = top > FP8_TINY;  // a block with nothing above that is held as zeros
  const float inv = held ? __fmul_rn(__frcp_rn(top), FP8_MAX) : 0.f;
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    float y[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      y[k] = __fmul_rn(x[j + k], inv);
      if (CHANCE && (had >> (j + k) & 1) && y[k] < 480.f) y[k] = round_by_chance(y[k], mix32(chance + j + k) >> 12);
      if (ROOT && x[j + k] > 0.f && y[k] < FP8_MIN) y[k] = FP8_MIN;
    }
    const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
    w[j >> 2] |= held ? c << (j & 2) * 8 : 0u;
  }
  if (vec && i + 8 <= n) {
    *reinterpret_cast<uint2*>(p + i) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) p[i + j] = (uint8_t)(w[j >> 2] >> (j & 3) * 8);
  }
  return held ? __fmul_rn(top, 1.f / FP8_MAX) : 0.f;
}

// CHANCE: the roots' codes are rounded by chance in this step (8 bits only).
template <bool EIGHT, bool GRAD_BF16, bool CHANCE, int CAP>
__device__ __forceinline__ void adam_blocks(const AdamTable<CAP>& tab, const AdamConst& c, bool scaled) {
  const int lane = threadIdx.x & 31;
  const int total = tab.before[tab.n];
  int k = 0;  // the tensor of the block at hand; blocks come in ascending order
  for (int b = blockIdx.x * ADAM_WARPS + (threadIdx.x >> 5); b < total; b += gridDim.x * ADAM_WARPS) {
    int hi = tab.n - 1;
    if (tab.before[k + 1] > b) hi = k;
    while (k < hi) {  // the last tensor with before <= b; those without elements have no blocks
      const int mid = (k + hi + 1) >> 1;
      if (tab.before[mid] <= b)
        k = mid;
      else
        hi = mid - 1;
    }
    const EpAdamWTensor& t = tab.t[k];
    const int64_t block = b - tab.before[k], i = block * ADAM_BLOCK + lane * 8, n = t.n;
    const bool vec = t.vec != 0;
    float p[8], g[8], m[8], v[8], root[8];
    uint32_t had = 0;
    load8((const float*)t.p, i, n, vec, p);
    if (GRAD_BF16)
      load8_bf16((const uint16_t*)t.g, i, n, vec, g);
    else
      load8((const float*)t.g, i, n, vec, g);
    if (EIGHT) {
      load8_codes((const uint8_t*)t.m, i, n, vec, t.m_scale[block], m);
      load8_codes((const uint8_t*)t.v, i, n, vec, t.v_scale[block], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (CHANCE) had |= v[j] > 0.f ? 1u << j : 0u;
        v[j] = __fmul_rn(v[j], v[j]);
      }
    } else {
      load8((const float*)t.m, i, n, vec, m);
      load8((const float*)t.v, i, n, vec, v);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) adam_element(c, scaled, p[j], g[j], m[j], v[j], root[j]);
    store8((float*)t.p, i, n, vec, p);
    if (t.copy) store8_bf16((uint16_t*)t.copy, i, n, vec, p);
    if (EIGHT) {
      // elements behind the tensor's end are 0 all along, and a 0 gradient keeps them so
      const float ms = store8_codes<false, false>((uint8_t*)t.m, i, n, vec, m, 0, 0);
      const uint32_t chance = CHANCE ? mix32(mix32(c.chance + (uint32_t)k) + (uint32_t)(i >> 3)) << 3 : 0u;
      const float vs = store8_codes<true, CHANCE>((uint8_t*)t.v, i, n, vec, root, chance, had);
      if (lane == 0) {
        t.m_scale[block] = ms;
        t.v_scale[block] = vs;
      }
    } else {
      store8((float*)t.m, i, n, vec, m);
      store8((float*)t.v, i, n, vec, v);
    }
  }
}

template <bool EIGHT, bool GRAD_BF16, int CAP>
__global__ void __launch_bounds__(ADAM_WARPS * 32, 4)
    k_adamw(const __grid_constant__ AdamTable<CAP> tab, const __grid_constant__ AdamArgs a) {
  __shared__ AdamConst s_c;
  wait_for_predecessor();
  if (threadIdx.x == 0) s_c = adam_const(a);
  __syncthreads();
  const AdamConst c = s_c;
  const bool scaled = a.grad_scale != nullptr;
  if (EIGHT && c.chance)
    adam_blocks<EIGHT, GRAD_BF16, EIGHT, CAP>(tab, c, scaled);
  else
    adam_blocks<EIGHT, GRAD_BF16, false, CAP>(tab, c, scaled);
}

template <int CAP>
static const void* adam_kernel(bool eight, bool grad_bf16) {
  return eight ? grad_bf16 ? (const void*)k_adamw<true, true, CAP> : (const void*)k_adamw<true, false, CAP>
               : grad_bf16 ? (const void*)k_adamw<false, true, CAP> : (const void*)k_adamw<false, false, CAP>;
}

}  // namespace ep

using namespace ep;

extern "C" int ep_adamw(const EpAdamWTensor* tensors, int n_tensors, int state_bits, int grad_dtype,
                        const int32_t* step, double lr, const float* lr_dev, double beta1, double beta2, double eps,
                        double weight_decay, const float* grad_scale, cudaStream_t stream) {
  if (n_tensors < 0 || (state_bits != 8 && state_bits != 32)) return EP_ERR_ARG;
  if (grad_dtype != EP_DTYPE_F32 && grad_dtype != EP_DTYPE_BF16) return EP_ERR_ARG;
  if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0 && eps >= 0.0) || !isfinite(eps) || !isfinite(lr) ||
      !isfinite(weight_decay))
    return EP_ERR_ARG;
  if (n_tensors == 0) return EP_OK;
  if (!tensors || !step || ((uintptr_t)step & 3) || ((uintptr_t)lr_dev & 3) || ((uintptr_t)grad_scale & 3))
    return EP_ERR_ARG;
  const bool eight = state_bits == 8, gb = grad_dtype == EP_DTYPE_BF16;
  const uintptr_t gmask = gb ? 1 : 3, smask = eight ? 0 : 3;
  for (int i = 0; i < n_tensors; ++i) {
    const EpAdamWTensor& t = tensors[i];
    if (t.n < 0 || (t.n + ADAM_BLOCK - 1) / ADAM_BLOCK >= ((int64_t)1 << 30)) return EP_ERR_ARG;
    if (t.n == 0) continue;
    if (!t.p || !t.g || !t.m || !t.v || (eight && (!t.m_scale || !t.v_scale))) return EP_ERR_ARG;
    if (((uintptr_t)t.p & 3) || ((uintptr_t)t.g & gmask) || ((uintptr_t)t.m & smask) || ((uintptr_t)t.v & smask) ||
        ((uintptr_t)t.copy & 1) || ((uintptr_t)t.m_scale & 3) || ((uintptr_t)t.v_scale & 3))
      return EP_ERR_ARG;
  }
  const AdamArgs a{lr, beta1, beta2, eps, weight_decay, lr_dev, grad_scale, step};
  AdamTable<ADAM_TENSORS> tab;
  int i = 0;
  while (i < n_tensors) {
    tab.n = 0;
    int64_t blocks = 0;
    for (; i < n_tensors && tab.n < ADAM_TENSORS; ++i) {
      EpAdamWTensor t = tensors[i];
      if (t.n == 0) continue;
      const int64_t more = (t.n + ADAM_BLOCK - 1) / ADAM_BLOCK;
      if (blocks + more >= ((int64_t)1 << 30)) break;
      t.vec = aligned16(t.p) && aligned16(t.g) && aligned16(t.copy) && aligned16(t.m) && aligned16(t.v);
      tab.before[tab.n] = (int32_t)blocks;
      tab.t[tab.n++] = t;
      blocks += more;
    }
    if (tab.n == 0) break;
    tab.before[tab.n] = (int32_t)blocks;
    // Many short rounds of CTAs rather than one resident grid: 100 M elements in 300 tensors 424 us against 496 with
    // 8 CTAs an SM in all (and 441 with them at 4 resident), 352 M with 8-bit moments 1047 against 1180
    const int64_t want = (blocks + ADAM_WARPS - 1) / ADAM_WARPS, most = (int64_t)num_sms() * 128;
    AdamTable<ADAM_FEW> few;
    const bool small = tab.n <= ADAM_FEW;
    if (small) {
      for (int k = 0; k < tab.n; ++k) {
        few.t[k] = tab.t[k];
        few.before[k] = tab.before[k];
      }
      few.before[tab.n] = tab.before[tab.n];
      few.n = tab.n;
    }
    const void* fn = small ? adam_kernel<ADAM_FEW>(eight, gb) : adam_kernel<ADAM_TENSORS>(eight, gb);
    void* args[] = {small ? (void*)&few : (void*)&tab, (void*)&a};
    if (launch_pdl(fn, dim3((unsigned)(want < most ? want : most)), dim3(ADAM_WARPS * 32), args, 0, stream) !=
        cudaSuccess)
      return EP_ERR_CUDA;
    count_launch();
  }
  return EP_OK;
}
