// The experts' products between dispatch and combine, and their gradients, over
// the slots of the dispatch buffer (home experts and replicas, each a run of
// consecutive rows): for every slot s with weights W of its expert
//   ep_expert_gemm         y_s = x_s W^T, or x_s W
//   ep_expert_up           h_s = silu(x_s Wg^T) * (x_s Wu^T)
//   ep_expert_up_backward  the gradient of that, from dy_s W2
//   ep_expert_wgrad        g_s = a_s^T b_s, fp32
//
// One persistent kernel per form, one CTA per SM, two CTAs (a cluster) on one
// tile: 256 rows by 512 columns in two accumulators (one of 256 in the weight
// gradient), of which each CTA holds half of the rows and half of each operand.
// Alone, a CTA with a 128 x 256 tile would read 12 KB of operands per product of
// 128 cycles and write as much for the next, more than the 128 bytes per cycle its
// shared memory takes; a pair shares the second operand and needs 8 KB each.  Two
// accumulators share the rows' operand too, so a quarter less comes from L2.  A
// pair walks output tiles in a fixed order; the slots' row counts are on the
// device, so every CTA first scans them into shared memory (tiles before each
// slot) and finds a tile's slot there by bisection (warp 2, some tiles ahead): no
// launch depends on a count the host would have to read.  In each CTA a thread of
// warp 0 brings operand tiles of 64 along the contraction into a ring in shared
// memory (TMA, 128-byte swizzle); one of the leader's warp 1 issues the tensor-core
// products into the accumulators in tensor memory; warps 4-11 take a finished
// accumulator into registers, give it back, and bring it through the epilogue to
// global memory while the next tile's products run.
//
// Measured (B200; one call at a time with a flush of L2 between, and in a loop over new inputs, where the power cap takes
// its part): first projection of 196,608 rows in 64 slots, H 2048, I 1024, its products kept, 1253 us = 1316 TFLOP/s, in a
// loop 1450 to 1540; weight gradient of the same 668 to 683 us = 1220, 800 to 850; second projection of 32,768 rows in 13
// slots, H 7168, I 2048, 757 us = 1270, 773 to 813; backward of the activation there 803 us = 1197, 930 to 970.  The
// library's product of one dense matrix of the second projection's size takes 627 us after a pause and 700 in a loop: a
// bound to compare with, not the same work.
//
// A tile's rows are its slot's rows from a multiple of 256 on; rows behind the
// slot's end belong to the next slot and only make accumulator rows that are
// not stored.  In the weight gradient the rows are the contraction: there the
// lines behind the slot's end are zeroed in shared memory (in both operands, so
// that an infinity or NaN of the next slot takes no part) by warp 3.
//
// The accumulator's additions cut off rather than round: over n rows of one sign
// the sum comes out up to n * 4.5e-9 too small (measured: 1.0e-5 at 4096 rows,
// 7.4e-5 at 16,384).  bf16 results do not see that; the weight gradient is fp32
// and may run over a hundred thousand rows, so it takes the accumulator out
// every 512 rows (6e-7 at most of one sign, whatever the slot's length) and adds
// these partial sums in registers.
#include <cuda.h>

#include "umma.cuh"

namespace ep {

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool encode_tiles(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                  const uint32_t* box) {
  static const EncodeTiled encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return (EncodeTiled)fn;
  }();
  if (!encode) return false;
  const cuuint32_t unit[3] = {1, 1, 1};
  cuuint64_t d[3], s[2];
  cuuint32_t b[3];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    if (i) s[i - 1] = strides[i - 1];
  }
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), d, s, b, unit,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int TM = 256, TN = 256, TK = 64;  // of a pair of CTAs; each has TM / 2 rows of A, TN / 2 of B
constexpr int EXP_THREADS = 384;
constexpr uint32_t A_BYTES = TM / 2 * TK * 2, B_BYTES = TN / 2 * TK * 2;
constexpr uint32_t RING_BYTES = 12 * A_BYTES;  // 4 stages of an A and two B tiles, or 6 of one each
constexpr int MAX_STAGES = 6;
constexpr int TILES_AHEAD = 4;
constexpr int SORTED_SLOTS = 512;
constexpr int PART = 8;  // WGRAD: blocks of TK rows that the accumulator sums by itself
constexpr int MAX_SLOTS = 2 * EP_MAX_EXPERTS + EP_MAX_RANKS - 1;  // E homes and E + R - 1 replicas
constexpr int MAX_IDS = EP_MAX_EXPERTS + MAX_SLOTS;  // ids of slots lie below n_w + n_rep, and n_rep alone may be MAX_SLOTS
constexpr int BAND = 8;  // tiles of a slot are walked in bands of 8 row blocks, so that the CTAs at work at a
                         // time share both operands in L2 (4 to 16 measured the same)

// What a product is made of: how B is held, and what happens to a finished tile.
enum Form { Y_NT, Y_NN, UP, UP_BACKWARD, WGRAD };

// Accumulators of TN columns that a tile takes at most, the stages that leaves
// in the ring, and the result's columns in one accumulator.
template <Form F>
struct Shape {
  static constexpr int halves = F == WGRAD ? 1 : 2;
  static constexpr uint32_t stage_bytes = A_BYTES + halves * B_BYTES;
  static constexpr int stages = RING_BYTES / stage_bytes;
  static constexpr int tn = F == UP ? TN / 2 : TN;
  static_assert(stages <= MAX_STAGES && RING_BYTES % stage_bytes == 0, "");
};

struct ExpertArgs {
  int64_t rows;
  int N, K;          // columns of the result (UP: of h), contraction (WGRAD: N columns, M = K rows of the result)
  int n_slots, n_w, n_rep;
  const int32_t *cu, *slots, *rep;
  uint16_t *y, *y2;  // Y: y; UP: h, gu or NULL; UP_BACKWARD: dgu, h or NULL
  const uint16_t* gu;
  float* g_home;
  void* g_rep;
  int64_t ld_home, ld_rep;  // elements between experts
  bool rep_bf16, add_home, add_rep;  // add: to what is there
  uint64_t wait_ns;  // the bound of a wait: a second, and more where a tile may take long
  int32_t* dev_status;
};

// Rows [begin, begin + len) of slot s and where its weights (or its gradient) are: w < n_w the expert of the
// weights; for WGRAD the slot id itself.  len < 0: no such slot, nothing to do.
struct Slot {
  int64_t begin;
  int len, w;
};

// The tables are read past L1: the kernel may start while the one that writes them ends.
template <Form F>
__device__ __forceinline__ Slot load_slot(const ExpertArgs& a, int s, int32_t* bits) {
  const int id = a.slots ? __ldcg(a.slots + s) : s;
  Slot r{0, -1, id};
  if (id < 0) return r;
  if (id >= a.n_w + a.n_rep || (id >= a.n_w && F != WGRAD && !a.rep)) {
    *bits |= EP_DEV_BAD_EXPERT_ID;
    return r;
  }
  if (F != WGRAD && id >= a.n_w) {
    r.w = __ldcg(a.rep + (id - a.n_w));
    if (r.w < 0 || r.w >= a.n_w) {
      *bits |= EP_DEV_BAD_EXPERT_ID;
      return r;
    }
  }
  const int b = __ldcg(a.cu + s), e = __ldcg(a.cu + s + 1);
  if (b < 0 || e < b || e > a.rows) {
    *bits |= EP_DEV_BAD_ROW;
    return r;
  }
  r.begin = b;
  r.len = e - b;
  return r;
}

// Consecutive slots share their ends, so they can only overlap behind an entry that is below the one before it.  Then a
// slot with rows that begins before the end of an earlier one (whose id and rows are good) is left out like one that
// does not fit: two slots would write the same rows, and tiles are counted for disjoint ones.
__device__ __forceinline__ bool descends(const ExpertArgs& a, int s) {
  return __ldcg(a.cu + s) > __ldcg(a.cu + s + 1);
}

template <Form F>
__device__ __forceinline__ bool overlaps(const ExpertArgs& a, int s) {
  int32_t ignore = 0;
  const Slot slot = load_slot<F>(a, s, &ignore);
  if (slot.len <= 0) return false;
  for (int o = 0; o < s; ++o) {
    const Slot other = load_slot<F>(a, o, &ignore);
    if (other.len > 0 && other.begin + other.len > slot.begin) return true;
  }
  return false;
}

struct Tile {
  Slot slot;
  int m, n;    // first row (within the slot; WGRAD: of the result) and column
  int halves;  // accumulators that it takes; 0: no columns left, not a tile
  int steps;   // blocks of TK along the contraction; -1: no tile any more
};

struct ExpertShared {
  uint4 turn[8][128];          // the epilogue warps' 32 rows of 64 bytes
  uint64_t full[MAX_STAGES];   // the leader's: both CTAs' operands of a stage are there
  uint64_t empty[MAX_STAGES];  // the products have read a stage
  uint64_t tail[MAX_STAGES];   // WGRAD: this CTA's operands of a slot's last stage are there, to be cut
  uint64_t acc_full[2];
  uint64_t acc_empty[2];       // the leader's: both CTAs have taken an accumulator out
  uint64_t tile_full[TILES_AHEAD], tile_empty[TILES_AHEAD];
  Tile tiles[TILES_AHEAD];     // found ahead by warp 2
  uint32_t tmem;
  int abort;
  int32_t warp_sums[32];
  uint16_t sorted[SORTED_SLOTS];  // WGRAD: the slots by descending rows
  uint32_t seen[(MAX_IDS + 31) / 32], twice[(MAX_IDS + 31) / 32];  // WGRAD: ids, and those that stand twice
  int32_t before[MAX_SLOTS + 1];  // tiles before each slot
};

// A thread's bounded wait, that gives up as soon as another role of the CTA has.
__device__ __forceinline__ bool wait_thread(uint64_t* bar, uint32_t parity, ExpertShared* sh, const ExpertArgs& a) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*(volatile int*)&sh->abort) return false;
    if (globaltimer_ns() - t0 > a.wait_ns) {
      *(volatile int*)&sh->abort = 1;
      flag(a.dev_status, EP_DEV_COPY_TIMEOUT);
      return false;
    }
  }
  return true;
}

// The same for a whole warp, with one outcome.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, ExpertShared* sh, const ExpertArgs& a) {
  return __all_sync(0xffffffffu, wait_thread(bar, parity, sh, a));
}

// The order of a pair's work: `wide` tiles of all the columns a tile can take,
// then `narrow` tiles of one accumulator each.  Where the last round of wide
// tiles would keep at most half of the pairs at work, it is done in halves by
// twice as many.
struct Order {
  int wide, narrow;
};

template <Form F>
__device__ __forceinline__ Order make_order(int total, int pairs) {
  const int last = total % pairs;
  if (Shape<F>::halves == 1 || 2 * last > pairs) return Order{total, 0};
  return Order{total - last, 2 * last};
}

template <Form F>
__device__ __forceinline__ Tile find_tile(const ExpertArgs& a, const ExpertShared* sh, const Order& o, int t,
                                          int* hint) {
  constexpr int tn = Shape<F>::tn, halves = Shape<F>::halves;
  const int half = t < o.wide ? -1 : (t - o.wide) & 1;
  if (half >= 0) t = o.wide + ((t - o.wide) >> 1);
  int lo = *hint, hi = a.n_slots - 1;  // the last slot with before[s] <= t; tiles come in ascending order
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sh->before[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  *hint = lo;
  int32_t ignore = 0;
  Tile r;
  r.slot = load_slot<F>(a, F == WGRAD && a.n_slots <= SORTED_SLOTS ? sh->sorted[lo] : lo, &ignore);
  const int nb = (a.N + halves * tn - 1) / (halves * tn);
  const int mb = ((F == WGRAD ? a.K : r.slot.len) + TM - 1) / TM;
  const int i = t - sh->before[lo];
  const int band = i / (BAND * nb), in_band = i - band * BAND * nb;
  const int height = min(BAND, mb - band * BAND);
  r.n = in_band / height * (halves * tn) + max(half, 0) * tn;
  r.m = (band * BAND + in_band % height) * TM;
  r.halves = r.n >= a.N ? 0 : half < 0 && halves == 2 && r.n + tn < a.N ? 2 : 1;
  r.steps = ((F == WGRAD ? r.slot.len : a.K) + TK - 1) / TK;
  return r;
}

// A role's walk over the tiles that warp 2 finds.  next() is false at the end, or
// when a wait ran out.  WARP: all lanes walk; otherwise one thread does.
template <bool WARP>
struct Walk {
  ExpertShared* sh;
  const ExpertArgs& a;
  int at;
  uint32_t phase;
  Tile tile;
  __device__ __forceinline__ Walk(ExpertShared* s, const ExpertArgs& args) : sh(s), a(args), at(0), phase(0) {}
  __device__ __forceinline__ bool next() {
    if (WARP) {
      if (!wait_warp(&sh->tile_full[at], phase, sh, a)) return false;
      tile = sh->tiles[at];
      __syncwarp();
    } else {
      if (!wait_thread(&sh->tile_full[at], phase, sh, a)) return false;
      tile = sh->tiles[at];
    }
    if (!WARP || (threadIdx.x & 31) == 0) mbar_arrive(&sh->tile_empty[at]);
    if (++at == TILES_AHEAD) {
      at = 0;
      phase ^= 1;
    }
    return tile.steps >= 0;
  }
};

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                    f32x2_to_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ void unpack8(uint4 p, float* v) {
  const uint32_t u[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_bits_to_f32(u[i] & 0xffffu);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// 1 / (1 + e^-g) by the hardware's 2^x and reciprocal (2^-22 and 2^-23 of themselves; the exponent |g| 2^-24): far
// inside bf16.  e^-g overflows to infinity for g below -88, where the result is 0.
__device__ __forceinline__ float sigmoid_fast(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504088896341f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}

// A warp's way between "a lane has a row" (as tensor memory gives it) and "four
// lanes have 64 bytes of a row" (as global memory wants it): 32 rows of 64 bytes
// in shared memory, its 16-byte units permuted so that neither side has bank
// conflicts.  Stored straight from the lanes, 16 bytes of 32 rows at a time, each
// 32-byte sector went out twice and the products waited for it (second projection
// of 32,768 rows 835 us against 771 us without any store).
struct Turn {
  uint4* buf;
  int lane, row, unit;  // row + 8 j and unit: this lane's place on the memory side
  __device__ __forceinline__ Turn(uint4* b, int l) : buf(b), lane(l), row(l >> 2), unit(l & 3) {}
  __device__ __forceinline__ uint4& mine(int u) { return buf[lane * 4 + (u ^ (lane >> 1 & 3))]; }
  __device__ __forceinline__ uint4& theirs(int j) {
    const int r = row + 8 * j;
    return buf[r * 4 + (unit ^ (r >> 1 & 3))];
  }
};

// 32 columns of bf16 (each lane its row's) to rows [0, rows) at to, columns below n
__device__ __forceinline__ void store_rows(Turn& t, const uint4* q, uint16_t* to, int64_t ld, int rows, int n) {
#pragma unroll
  for (int u = 0; u < 4; ++u) t.mine(u) = q[u];
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (t.row + 8 * j < rows && t.unit * 8 < n) st_v4(to + (t.row + 8 * j) * ld + t.unit * 8, t.theirs(j));
  __syncwarp();
}

__device__ __forceinline__ void store_rows(Turn& t, const float* v, uint16_t* to, int64_t ld, int rows, int n) {
  uint4 q[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) q[u] = pack8(v + 8 * u);
  store_rows(t, q, to, ld, rows, n);
}

// The other way in two steps, so that the loads can be under way early.  The results may go where these rows come from:
// a lane then stores what it has loaded itself (Turn gives it the same rows and unit both ways).
__device__ __forceinline__ void fetch_rows(const Turn& t, uint4* p, const uint16_t* from, int64_t ld, int rows, int n) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    p[j] = make_uint4(0, 0, 0, 0);
    if (t.row + 8 * j < rows && t.unit * 8 < n) p[j] = ld_once_v4(from + (t.row + 8 * j) * ld + t.unit * 8);
  }
}

__device__ __forceinline__ void turn_rows(Turn& t, const uint4* p, uint4* q) {
#pragma unroll
  for (int j = 0; j < 4; ++j) t.theirs(j) = p[j];
  __syncwarp();
#pragma unroll
  for (int u = 0; u < 4; ++u) q[u] = t.mine(u);
  __syncwarp();
}

// 32 columns of an expert's gradient: fp32 sixteen at a time, or bf16
__device__ __forceinline__ void store_grad(Turn& t, const ExpertArgs& a, int id, int64_t at, const float* v, int rows,
                                           int n) {
  const bool home = id < a.n_w;
  if (home || !a.rep_bf16) {
    float* to = (home ? a.g_home + (int64_t)id * a.ld_home : (float*)a.g_rep + (int64_t)(id - a.n_w) * a.ld_rep) + at;
#pragma unroll
    for (int c = 0; c < 32; c += 16) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float* x = v + c + 4 * u;
        t.mine(u) = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                               __float_as_uint(x[3]));
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (t.row + 8 * j < rows && c + t.unit * 4 < n) {
          float* q = to + (int64_t)(t.row + 8 * j) * a.N + c + t.unit * 4;
          uint4 s = t.theirs(j);
          if (home ? a.add_home : a.add_rep) {
            const float4 o = *reinterpret_cast<const float4*>(q);
            s = make_uint4(__float_as_uint(o.x + __uint_as_float(s.x)), __float_as_uint(o.y + __uint_as_float(s.y)),
                           __float_as_uint(o.z + __uint_as_float(s.z)), __float_as_uint(o.w + __uint_as_float(s.w)));
          }
          st_v4(q, s);
        }
      __syncwarp();
    }
  } else {
    uint16_t* to = (uint16_t*)a.g_rep + (int64_t)(id - a.n_w) * a.ld_rep + at;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (a.add_rep && t.row + 8 * j < rows && t.unit * 8 < n)
        t.theirs(j) = *reinterpret_cast<const uint4*>(to + (int64_t)(t.row + 8 * j) * a.N + t.unit * 8);
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float o[8];
      unpack8(t.mine(u), o);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = a.add_rep ? o[i] + v[8 * u + i] : v[8 * u + i];
      t.mine(u) = pack8(o);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (t.row + 8 * j < rows && t.unit * 8 < n)
        st_v4(to + (int64_t)(t.row + 8 * j) * a.N + t.unit * 8, t.theirs(j));
    __syncwarp();
  }
}

template <Form F>
__global__ void __launch_bounds__(EXP_THREADS, 1) __cluster_dims__(2, 1, 1)
    k_experts(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
              const __grid_constant__ ExpertArgs a) {
  extern __shared__ uint8_t s_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~(uintptr_t)1023);
  ExpertShared* sh = reinterpret_cast<ExpertShared*>(ring + RING_BYTES);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)pair_rank(), first = blockIdx.x >> 1, step = gridDim.x >> 1;
  constexpr int tn = Shape<F>::tn, halves = Shape<F>::halves, stages = Shape<F>::stages;
  constexpr uint32_t stage_bytes = Shape<F>::stage_bytes;

  if (tid == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&sh->full[i], 2);
      mbar_init(&sh->empty[i], 1);
      mbar_init(&sh->tail[i], 1);
    }
    for (int i = 0; i < TILES_AHEAD; ++i) {
      mbar_init(&sh->tile_full[i], 1);
      mbar_init(&sh->tile_empty[i], 9 + (rank == 0) + (F == WGRAD));  // warps 0 and 4-11, 1 of the leader, 3
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->acc_full[i], 1);
      mbar_init(&sh->acc_empty[i], 2 * 8);
    }
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc(&sh->tmem, 2 * TN);
  wait_for_predecessor();
  int32_t bits = 0;
  {
    // A weight gradient's tiles take as long as their slot has rows, and a pair takes every so many-th tile: with the
    // slots by descending rows, and every other round of tiles handed out backwards, all pairs get about the same
    // (196,608 rows in 64 slots of unlike length: 724 us against 767).  Every CTA finds the same order: ties by the slot.
    // Ranking each slot against all others is quick up to some hundred slots; longer tables stay as they are.
    const bool sorted = F == WGRAD && a.n_slots <= SORTED_SLOTS;
    if (F == WGRAD) {
      for (int i = tid; i < (MAX_IDS + 31) / 32; i += EXP_THREADS) sh->seen[i] = sh->twice[i] = 0;
      __syncthreads();
      for (int s = tid; s < a.n_slots; s += EXP_THREADS) {
        const Slot slot = load_slot<F>(a, s, &bits);
        if (slot.len < 0) continue;
        const uint32_t bit = 1u << (slot.w & 31);
        if (atomicOr(&sh->seen[slot.w >> 5], bit) & bit) atomicOr(&sh->twice[slot.w >> 5], bit);
      }
      __syncthreads();
    }
    if (sorted) {
      for (int s = tid; s < a.n_slots; s += EXP_THREADS) sh->before[s] = load_slot<F>(a, s, &bits).len;
      __syncthreads();
      for (int s = tid; s < a.n_slots; s += EXP_THREADS) {
        const int len = sh->before[s];
        int r = 0;
        for (int o = 0; o < a.n_slots; ++o) r += sh->before[o] > len || (sh->before[o] == len && o < s);
        sh->sorted[r] = (uint16_t)s;
      }
      __syncthreads();
    }
    const int nb = (a.N + halves * tn - 1) / (halves * tn);
    bool down = false;
    for (int s = tid; s < a.n_slots; s += EXP_THREADS) {
      down |= descends(a, s);
      const Slot slot = load_slot<F>(a, sorted ? sh->sorted[s] : s, &bits);
      int mb = slot.len < 0 ? 0 : ((F == WGRAD ? a.K : slot.len) + TM - 1) / TM;
      if (F == WGRAD && mb && (sh->twice[slot.w >> 5] >> (slot.w & 31) & 1)) {
        bits |= EP_DEV_BAD_EXPERT_ID;
        mb = 0;
      }
      if (F == WGRAD && slot.len == 0 && (slot.w < a.n_w ? a.add_home : a.add_rep)) mb = 0;  // nothing to add
      sh->before[s] = mb * nb;
    }
    if (__syncthreads_or(down)) {
      for (int s = tid; s < a.n_slots; s += EXP_THREADS)
        if (overlaps<F>(a, sorted ? sh->sorted[s] : s)) {
          bits |= EP_DEV_BAD_ROW;
          sh->before[s] = 0;
        }
    }
  }
  if (bits && blockIdx.x == 0) flag(a.dev_status, bits);
  umma_fence_before();
  __syncthreads();
  umma_fence_after();
  const int total = block_scan_array(sh->before, a.n_slots, sh->warp_sums);
  const Order order = make_order<F>(total, step);
  const uint32_t tmem = sh->tmem;
  pair_sync();  // the other CTA's barriers are set up

  if (tid == 0) {
    // ---- this CTA's operand tiles into the ring
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    Walk<false> walk(sh, a);
    while (ok && walk.next()) {
      const Tile& tile = walk.tile;
      // rows behind the slot's end need not be read where a whole half is
      const bool rows = F == WGRAD || tile.m + rank * (TM / 2) < tile.slot.len;
      const uint32_t bytes = tile.halves * B_BYTES + (rows ? A_BYTES : 0);
      for (int k = 0; k < tile.steps; ++k) {
        if (!(ok = wait_thread(&sh->empty[stage], phase ^ 1, sh, a))) break;
        uint8_t* sa = ring + stage * stage_bytes;
        uint8_t* sb = sa + A_BYTES;
        const int kk = k * TK;
        const bool tail = F == WGRAD && kk + TK > tile.slot.len;
        const uint32_t bar = tail ? smem_addr(&sh->tail[stage]) : leader_addr(&sh->full[stage]);
        pair_arrive_expect_tx(bar, bytes);
        if (F == WGRAD) {
          const int row = (int)tile.slot.begin + kk;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            tma_tile_2d(sa + i * 8192, &map_a, bar, tile.m + rank * (TM / 2) + i * 64, row);
            tma_tile_2d(sb + i * 8192, &map_b, bar, tile.n + rank * (TN / 2) + i * 64, row);
          }
        } else {
          if (rows) tma_tile_2d(sa, &map_a, bar, kk, (int)tile.slot.begin + tile.m + rank * (TM / 2));
#pragma unroll
          for (int h = 0; h < halves; ++h, sb += B_BYTES) {
            if (h >= tile.halves) break;
            const int n = tile.n + h * tn;
            if (F == UP) {  // the leader holds the gate's rows, the other CTA the up projection's
              tma_tile_3d(sb, &map_b, bar, kk, rank * a.N + n, tile.slot.w);
            } else if (F == Y_NT) {
              tma_tile_3d(sb, &map_b, bar, kk, n + rank * (TN / 2), tile.slot.w);
            } else {
              tma_tile_3d(sb, &map_b, bar, n + rank * (TN / 2), kk, tile.slot.w);
              tma_tile_3d(sb + 8192, &map_b, bar, n + rank * (TN / 2) + 64, kk, tile.slot.w);
            }
          }
        }
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  } else if (tid == 32 && rank == 0) {
    // ---- tensor-core products, issued by one thread: what stands between two issues is time the cores idle
    constexpr bool a_m = F == WGRAD, b_n = F == WGRAD || F == Y_NN || F == UP_BACKWARD;
    constexpr uint32_t idesc = umma_idesc(TM, TN, a_m, b_n);
    const uint32_t s0 = smem_addr(ring);
    const uint64_t da0 = a_m ? umma_smem_desc(s0, 8192, 1024) : umma_smem_desc(s0, 16, 1024);
    const uint64_t db0 = b_n ? umma_smem_desc(s0 + A_BYTES, 8192, 1024) : umma_smem_desc(s0 + A_BYTES, 16, 1024);
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    Walk<false> walk(sh, a);
    while (ok && walk.next()) {
      const Tile& tile = walk.tile;
      const bool two = halves == 2 && tile.halves == 2;
      for (int k = 0; k < tile.steps; ++k) {
        const int part = F == WGRAD ? k % PART : k;
        const bool last = k + 1 == tile.steps || (F == WGRAD && part + 1 == PART);
        if (part == 0 && !(ok = wait_thread(&sh->acc_empty[acc], acc_phase ^ 1, sh, a))) break;
        if (!(ok = wait_thread(&sh->full[stage], phase, sh, a))) break;
        umma_fence_after();
        const uint64_t da = da0 + (uint32_t)stage * (stage_bytes >> 4), db = db0 + (uint32_t)stage * (stage_bytes >> 4);
#pragma unroll
        for (int i = 0; i < TK / 16; ++i)  // 16 elements on: 32 bytes along K, two groups of 8 lines otherwise
          umma_bf16(tmem + acc * TN, da + (a_m ? i * 128 : i * 2), db + (b_n ? i * 128 : i * 2), idesc,
                    part > 0 || i > 0);
        if (last) umma_commit(&sh->acc_full[acc]);
        if (two) {
          // the next accumulator, which may be the first of its round
          if (part == 0) {
            if (!(ok = wait_thread(&sh->acc_empty[acc ^ 1], acc_phase ^ 1 ^ acc, sh, a))) break;
            umma_fence_after();
          }
#pragma unroll
          for (int i = 0; i < TK / 16; ++i)
            umma_bf16(tmem + (acc ^ 1) * TN, da + (a_m ? i * 128 : i * 2),
                      db + (B_BYTES >> 4) + (b_n ? i * 128 : i * 2), idesc, part > 0 || i > 0);
          if (last) umma_commit(&sh->acc_full[acc ^ 1]);
        }
        umma_commit(&sh->empty[stage]);
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
        if (last) {  // on by the accumulators taken: two bring the same one around again
          if (two)
            acc_phase ^= 1;
          else if (++acc == 2)
            acc = 0, acc_phase ^= 1;
        }
      }
    }
  } else if (warp == 2) {
    // ---- the tiles, a few ahead of the other warps: a search and loads that depend on each other
    int hint = 0, at = 0;
    uint32_t phase = 0;
    for (int i = 0;; ++i) {
      if (!wait_warp(&sh->tile_empty[at], phase ^ 1, sh, a)) break;
      Tile tile = {};
      tile.steps = -1;
      tile.halves = 1;
      const int t = i * step + (F == WGRAD && (i & 1) ? step - 1 - first : first);
      if (t < order.wide + order.narrow) tile = find_tile<F>(a, sh, order, t, &hint);
      else if (F == WGRAD && i * step < order.wide) continue;  // nothing in a last round that is handed out backwards
      if (tile.halves == 0) continue;
      if (lane == 0) {
        sh->tiles[at] = tile;
        mbar_arrive(&sh->tile_full[at]);
      }
      __syncwarp();
      if (tile.steps < 0) break;
      if (++at == TILES_AHEAD) {
        at = 0;
        phase ^= 1;
      }
    }
  } else if (F == WGRAD && warp == 3) {
    // ---- zero the lines behind a slot's end in its last block of rows
    int block = 0;  // blocks of rows so far, modulo the stages
    uint32_t phases = 0;
    Walk<true> walk(sh, a);
    while (walk.next()) {
      const Tile& tile = walk.tile;
      block = (block + tile.steps) % stages;
      const int valid = tile.slot.len % TK;
      if (valid == 0) continue;
      const int stage = (block + stages - 1) % stages;
      if (!wait_warp(&sh->tail[stage], phases >> stage & 1, sh, a)) break;
      phases ^= 1u << stage;
      uint8_t* s = ring + stage * stage_bytes;
      for (int i = lane; i < (TK - valid) * 8; i += 32) {
#pragma unroll
        for (int c = 0; c < (int)stage_bytes / 8192; ++c)
          *reinterpret_cast<uint4*>(s + c * 8192 + valid * 128 + i * 16) = make_uint4(0, 0, 0, 0);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) pair_arrive_release(leader_addr(&sh->full[stage]));
    }
  } else if (warp >= 4) {
    // ---- finished tiles to global memory: warp = 32 rows of this CTA's half, half of its columns
    const int row = (warp & 3) * 32;
    const int col = warp >= 8 ? tn / 2 : 0;
    const uint32_t lanes = (uint32_t)row << 16;  // the address's high half
    Turn turn(sh->turn[warp - 4], lane);
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    Walk<true> walk(sh, a);
    while (ok && walk.next()) {
      const Tile& tile = walk.tile;
      const int m = tile.m + rank * (TM / 2) + row;
      const int rows = (F == WGRAD ? a.K : tile.slot.len) - m;  // of this warp's 32, those that are stored
      if (F == WGRAD) {
        float sum[TN / 2];
#pragma unroll
        for (int i = 0; i < TN / 2; ++i) sum[i] = 0.f;
        for (int k = 0; k < tile.steps; k += PART) {
          if (!(ok = wait_warp(&sh->acc_full[acc], acc_phase, sh, a))) break;
          umma_fence_after();
#pragma unroll
          for (int c = 0; c < TN / 2; c += 16) {
            uint32_t r[16];
            tmem_load(tmem + lanes + acc * TN + col + c, r);
            tmem_wait_load(r);
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[c + i] += __uint_as_float(r[i]);
          }
          umma_fence_before();
          __syncwarp();
          if (lane == 0) pair_arrive(leader_addr(&sh->acc_empty[acc]));
          if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1;
          }
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < TN / 2; c += 32) {
          const int n = tile.n + col + c;
          if (n < a.N) store_grad(turn, a, tile.slot.w, (int64_t)m * a.N + n, sum + c, rows, a.N - n);
        }
      } else {
        const int64_t at = tile.slot.begin + m;
        for (int h = 0; ok && h < tile.halves; ++h) {
          const int n = tile.n + h * tn + col;
          const bool any = rows > 0 && n < a.N;  // the same for the whole warp
          const uint32_t src = tmem + lanes + acc * TN + col;
          const uint32_t free = leader_addr(&sh->acc_empty[acc]);
          uint4 g[4], w[4];
          if (F == UP_BACKWARD && any) {
            fetch_rows(turn, g, a.gu + at * 2 * a.N + n, 2 * a.N, rows, a.N - n);
            fetch_rows(turn, w, a.gu + at * 2 * a.N + a.N + n, 2 * a.N, rows, a.N - n);
          }
          if (!(ok = wait_warp(&sh->acc_full[acc], acc_phase, sh, a))) break;
          umma_fence_after();
          if (!any) {
            __syncwarp();
            if (lane == 0) pair_arrive(free);
          } else if (F == UP_BACKWARD) {
            uint32_t v[2][32];
#pragma unroll
            for (int c = 0; c < TN / 2; c += 32) {
              if (c % 64 == 0) {
                tmem_load(src + c, v[0]);
                tmem_load(src + c + 32, v[1]);
                tmem_wait_load(v[0]);
                tmem_wait_load(v[1]);
                if (c) {
                  umma_fence_before();
                  __syncwarp();
                  if (lane == 0) pair_arrive(free);
                }
              }
              uint4 qg[4], qw[4], qh[4];
              turn_rows(turn, g, qg);
              turn_rows(turn, w, qw);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float dg[8], du[8], h8[8];
                unpack8(qg[i], dg);
                unpack8(qw[i], du);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const float dh = __uint_as_float(v[c / 32 % 2][8 * i + j]);
                  const float sg = sigmoid_fast(dg[j]), si = dg[j] * sg;
                  h8[j] = si * du[j];
                  dg[j] = dh * du[j] * (sg + si * (1.f - sg));
                  du[j] = dh * si;
                }
                qg[i] = pack8(dg);
                qw[i] = pack8(du);
                qh[i] = pack8(h8);
              }
              const int nc = n + c;
              if (c + 32 < TN / 2) {
                fetch_rows(turn, g, a.gu + at * 2 * a.N + nc + 32, 2 * a.N, rows, a.N - nc - 32);
                fetch_rows(turn, w, a.gu + at * 2 * a.N + a.N + nc + 32, 2 * a.N, rows, a.N - nc - 32);
              }
              store_rows(turn, qg, a.y + at * 2 * a.N + nc, 2 * a.N, rows, a.N - nc);
              store_rows(turn, qw, a.y + at * 2 * a.N + a.N + nc, 2 * a.N, rows, a.N - nc);
              if (a.y2) store_rows(turn, qh, a.y2 + at * a.N + nc, a.N, rows, a.N - nc);
            }
          } else {
            // all of it into registers first: the products wait for the accumulator, not for the stores
            uint32_t v[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c)  // UP: the gate's 64 columns, then the up projection's
              tmem_load(src + (F == UP && c >= 2 ? TN / 2 + (c - 2) * 32 : c * 32), v[c]);
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_wait_load(v[c]);
            umma_fence_before();
            __syncwarp();
            if (lane == 0) pair_arrive(free);
#pragma unroll
            for (int c = 0; c < tn / 2; c += 32) {
              const int nc = n + c;
              float* x = reinterpret_cast<float*>(v[c / 32]);
              if (F != UP) {
                store_rows(turn, x, a.y + at * a.N + nc, a.N, rows, a.N - nc);
              } else {
                float* u = reinterpret_cast<float*>(v[c / 32 + 2]);
                if (a.y2) {
                  store_rows(turn, x, a.y2 + at * 2 * a.N + nc, 2 * a.N, rows, a.N - nc);
                  store_rows(turn, u, a.y2 + at * 2 * a.N + a.N + nc, 2 * a.N, rows, a.N - nc);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = x[i] * sigmoid_fast(x[i]) * u[i];
                store_rows(turn, x, a.y + at * a.N + nc, a.N, rows, a.N - nc);
              }
            }
          }
          if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1;
          }
        }
      }
    }
  }
  __syncwarp();
  umma_fence_before();
  __syncthreads();
  umma_fence_after();
  if (sh->abort && tid == 0) {
    // a wait ran out: give copies and products in flight time to land before the memory is given back
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < WAIT_LIMIT_NS / 10) {
    }
  }
  __syncthreads();
  pair_sync();  // nothing of the other CTA's reaches for this one's shared or tensor memory any more
  if (warp == 2) tmem_free(tmem, 2 * TN);
}

constexpr size_t EXP_SMEM = 1024 + RING_BYTES + sizeof(ExpertShared);

// ---------------------------------------------------------------- few rows
//
// Decoding: a few rows to a slot, the time is that of reading the weights.  The
// tiles above would multiply 256 rows for the sake of three (at 192 rows over 64
// experts, H 2048, I 1024, up: 104 us, the weights alone 82).  Here the weights are
// the operand with 128 rows and up to 32 of the slot's rows are the columns: a
// product of 128 x 32, and a tile is two of them (UP: 128 rows of the gate and of
// the up projection; otherwise 256 rows of W) with fresh weights for nearly all of
// what is loaded (90 us there).  One CTA to a tile, 160 KB of weights on the way to
// each SM.
constexpr int FEW = 32;  // rows of a slot to a tile
constexpr int FEW_THREADS = 256, FEW_STAGES = 5;
constexpr uint32_t FEW_W = 128 * TK * 2, FEW_X = FEW * TK * 2, FEW_STAGE = 2 * FEW_W + FEW_X;

struct FewShared {
  uint64_t full[FEW_STAGES], empty[FEW_STAGES], acc_full[2], acc_empty[2];
  uint32_t tmem;
  int abort;
  int32_t warp_sums[32];
  int32_t before[MAX_SLOTS + 1];
};

constexpr size_t FEW_SMEM = 1024 + FEW_STAGES * FEW_STAGE + sizeof(FewShared);

// Same walk in every role (tiles are few): the slot by bisection, then its blocks of rows, the weights' blocks outermost.
template <Form F>
__device__ __forceinline__ Tile find_few(const ExpertArgs& a, const FewShared* sh, int t, int* hint) {
  int lo = *hint, hi = a.n_slots - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sh->before[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  *hint = lo;
  int32_t ignore = 0;
  Tile r;
  r.slot = load_slot<F>(a, lo, &ignore);
  const int mb = (r.slot.len + FEW - 1) / FEW, i = t - sh->before[lo];
  r.n = i / mb * (F == UP ? 128 : 256);
  r.m = i % mb * FEW;
  r.halves = F == UP || r.n + 128 < a.N ? 2 : 1;
  r.steps = (a.K + TK - 1) / TK;
  return r;
}

__device__ __forceinline__ bool wait_few(uint64_t* bar, uint32_t parity, FewShared* sh, const ExpertArgs& a) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*(volatile int*)&sh->abort) return false;
    if (globaltimer_ns() - t0 > a.wait_ns) {
      *(volatile int*)&sh->abort = 1;
      flag(a.dev_status, EP_DEV_COPY_TIMEOUT);
      return false;
    }
  }
  return true;
}

template <Form F>
__global__ void __launch_bounds__(FEW_THREADS, 1)
    k_experts_few(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                  const __grid_constant__ ExpertArgs a) {
  static_assert(F == UP || F == Y_NT, "");
  extern __shared__ uint8_t s_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~(uintptr_t)1023);
  FewShared* sh = reinterpret_cast<FewShared*>(ring + FEW_STAGES * FEW_STAGE);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int tn = F == UP ? 128 : 256;

  if (tid == 0) {
    for (int i = 0; i < FEW_STAGES; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->acc_full[i], 1);
      mbar_init(&sh->acc_empty[i], 4);
    }
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc_alone(&sh->tmem, 4 * FEW);  // two tiles' accumulators
  wait_for_predecessor();
  int32_t bits = 0;
  {
    const int nb = (a.N + tn - 1) / tn;
    bool down = false;
    for (int s = tid; s < a.n_slots; s += FEW_THREADS) {
      down |= descends(a, s);
      const Slot slot = load_slot<F>(a, s, &bits);
      sh->before[s] = slot.len <= 0 ? 0 : (slot.len + FEW - 1) / FEW * nb;
    }
    if (__syncthreads_or(down)) {
      for (int s = tid; s < a.n_slots; s += FEW_THREADS)
        if (overlaps<F>(a, s)) {
          bits |= EP_DEV_BAD_ROW;
          sh->before[s] = 0;
        }
    }
  }
  if (bits && blockIdx.x == 0) flag(a.dev_status, bits);
  umma_fence_before();
  __syncthreads();
  umma_fence_after();
  const int total = block_scan_array(sh->before, a.n_slots, sh->warp_sums);
  const uint32_t tmem = sh->tmem;

  if (tid == 0) {
    int stage = 0, hint = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      const Tile tile = find_few<F>(a, sh, t, &hint);
      for (int k = 0; k < tile.steps; ++k) {
        if (!(ok = wait_few(&sh->empty[stage], phase ^ 1, sh, a))) break;
        uint8_t* s = ring + stage * FEW_STAGE;
        uint64_t* bar = &sh->full[stage];
        mbar_arrive_expect_tx(bar, tile.halves * FEW_W + FEW_X);
        const int kk = k * TK;
        tma_tile_3d_alone(s, &map_w, bar, kk, tile.n, tile.slot.w);
        if (tile.halves == 2)
          tma_tile_3d_alone(s + FEW_W, &map_w, bar, kk, F == UP ? a.N + tile.n : tile.n + 128, tile.slot.w);
        tma_tile_2d_alone(s + 2 * FEW_W, &map_x, bar, kk, (int)tile.slot.begin + tile.m);
        if (++stage == FEW_STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  } else if (tid == 32) {
    constexpr uint32_t idesc = umma_idesc(128, FEW, false, false);
    int stage = 0, hint = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      const Tile tile = find_few<F>(a, sh, t, &hint);
      if (!(ok = wait_few(&sh->acc_empty[acc], acc_phase ^ 1, sh, a))) break;
      for (int k = 0; k < tile.steps; ++k) {
        if (!(ok = wait_few(&sh->full[stage], phase, sh, a))) break;
        umma_fence_after();
        const uint32_t s = smem_addr(ring + stage * FEW_STAGE);
        const uint64_t dx = umma_smem_desc(s + 2 * FEW_W, 16, 1024);
        for (int h = 0; h < tile.halves; ++h) {
          const uint64_t dw = umma_smem_desc(s + h * FEW_W, 16, 1024);
#pragma unroll
          for (int i = 0; i < TK / 16; ++i)
            umma_bf16_alone(tmem + (2 * acc + h) * FEW, dw + i * 2, dx + i * 2, idesc, k > 0 || i > 0);
        }
        umma_commit_alone(&sh->empty[stage]);
        if (++stage == FEW_STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (ok) umma_commit_alone(&sh->acc_full[acc]);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
  } else if (warp >= 4) {
    // lane = column of the result: 32 neighbouring columns of a row go out together
    const int col = (warp - 4) * 32 + lane;
    int hint = 0, acc = 0;
    uint32_t acc_phase = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
      const Tile tile = find_few<F>(a, sh, t, &hint);
      if (!__all_sync(0xffffffffu, wait_few(&sh->acc_full[acc], acc_phase, sh, a))) break;
      umma_fence_after();
      const uint32_t src = tmem + ((uint32_t)(warp - 4) << 21) + 2 * acc * FEW;
      uint32_t r[2][FEW];
      tmem_load(src, r[0]);
      tmem_load(src + FEW, r[1]);  // not written where the tile has one half; then it is not used either
      tmem_wait_load(r[0]);
      tmem_wait_load(r[1]);
      umma_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->acc_empty[acc]);
      const int rows = tile.slot.len - tile.m, n = tile.n + col;
      const int64_t at = tile.slot.begin + tile.m;
#pragma unroll
      for (int i = 0; i < FEW; ++i) {
        if (i >= rows) break;
        const float v = __uint_as_float(r[0][i]), u = __uint_as_float(r[1][i]);
        if (F == UP) {
          if (n < a.N) {
            a.y[(at + i) * a.N + n] = (uint16_t)f32x2_to_bf16x2(v * sigmoid_fast(v) * u, 0.f);
            if (a.y2) {
              uint16_t* gu = a.y2 + (at + i) * 2 * a.N + n;
              gu[0] = (uint16_t)f32x2_to_bf16x2(v, 0.f);
              gu[a.N] = (uint16_t)f32x2_to_bf16x2(u, 0.f);
            }
          }
        } else {
          if (n < a.N) a.y[(at + i) * a.N + n] = (uint16_t)f32x2_to_bf16x2(v, 0.f);
          if (n + 128 < a.N) a.y[(at + i) * a.N + n + 128] = (uint16_t)f32x2_to_bf16x2(u, 0.f);
        }
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
  }
  __syncwarp();
  umma_fence_before();
  __syncthreads();
  umma_fence_after();
  if (sh->abort && tid == 0) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < WAIT_LIMIT_NS / 10) {
    }
  }
  __syncthreads();
  if (warp == 2) tmem_free_alone(tmem, 4 * FEW);
}

// A warp may wait for as long as a tile takes, and a slot of the weight gradient may have a thousand million rows: 2 us
// for each block of the contraction (64 KB, at most 0.8 us where all SMs read from HBM) on top of a second.
template <Form F>
static uint64_t wait_bound(const ExpertArgs& a) {
  return WAIT_LIMIT_NS + (uint64_t)(F == WGRAD ? a.rows : (int64_t)a.K) / TK * 2000;
}

template <Form F>
static int launch_few(const CUtensorMap& mx, const CUtensorMap& mw, ExpertArgs a, cudaStream_t stream) {
  a.wait_ns = wait_bound<F>(a);
  if (!raise_smem_limit((const void*)k_experts_few<F>, FEW_SMEM)) return EP_ERR_CUDA;
  void* args[] = {(void*)&mx, (void*)&mw, (void*)&a};
  if (launch_pdl((const void*)k_experts_few<F>, dim3(num_sms()), dim3(FEW_THREADS), args, FEW_SMEM, stream) !=
      cudaSuccess)
    return EP_ERR_CUDA;
  count_launch();
  return EP_OK;
}

// Few rows to a slot on average: then the weights' bytes are what counts.  Rows spread evenly, us wide / few:
//   up, 64 experts, H 2048, I 1024      1 to 8 rows a slot 100 / 90   32: 102 / 92   64: 104 / 109
//   second projection of the same                1 to 8: 55 / 53          32: 57 / 55    64: 59 / 72
//   8 experts, H 7168, I 2048                    1 to 8: 55 / 47 to 49    32: 55 / 51    64: 57 / 74
//   64 experts, H 7168, I 2048                   1 to 8: 305 to 315 / 274 to 283  32: 324 / 291  64: 330 / 420
// The host knows the average only.  With all rows in one slot an average of 8 costs nothing or little in the first three
// (up 26 / 26; 18 / 18; 23 / 27) and 25 / 74 in the last (512 rows of one expert), one of 16 costs 29 / 49, 18 / 27, 25 / 27
// and 35 / 123: so up to 8.  The other forms have no such variant.
static bool few_rows(int64_t rows, int n_slots, int n_w) { return rows <= 8 * (int64_t)(n_slots < n_w ? n_slots : n_w); }

template <Form F>
static int launch_experts(const CUtensorMap& ma, const CUtensorMap& mb, ExpertArgs a, cudaStream_t stream) {
  a.wait_ns = wait_bound<F>(a);
  if (!raise_smem_limit((const void*)k_experts<F>, EXP_SMEM)) return EP_ERR_CUDA;
  void* args[] = {(void*)&ma, (void*)&mb, (void*)&a};
  if (launch_pdl((const void*)k_experts<F>, dim3(num_sms() / 2 * 2), dim3(EXP_THREADS), args, EXP_SMEM, stream) !=
      cudaSuccess)
    return EP_ERR_CUDA;
  count_launch();
  return EP_OK;
}

// x as tiles of 64 columns and W, rows x cols per expert, along K or along N.
static bool map_rows(CUtensorMap* m, const void* p, int64_t rows, int cols, int box_rows) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, strides[1] = {(uint64_t)cols * 2};
  const uint32_t box[2] = {64, (uint32_t)box_rows};
  return encode_tiles(m, p, 2, dims, strides, box);
}

static bool map_weights(CUtensorMap* m, const void* p, int n, int rows, int cols, int box_rows) {
  const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)n};
  const uint64_t strides[2] = {(uint64_t)cols * 2, (uint64_t)rows * cols * 2};
  const uint32_t box[3] = {64, (uint32_t)box_rows, 1};
  return encode_tiles(m, p, 3, dims, strides, box);
}

static bool valid_slots(int64_t rows, int n_w, const int32_t* cu, int n_slots, int n_rep) {
  return rows >= 0 && rows < ((int64_t)1 << 31) - 1024 && n_w >= 1 && n_w <= EP_MAX_EXPERTS && n_slots >= 0 &&
         n_slots <= MAX_SLOTS && n_rep >= 0 && n_rep <= MAX_SLOTS && (n_slots == 0 || cu);
}

// Widths are multiples of 8 (16-byte rows) and small enough that a coordinate, or 2 * width, fits 31 bits with room.
static bool valid_width(int64_t n) { return n >= 8 && n % 8 == 0 && n <= (1 << 28); }

// Tiles of a call fit 31 bits, and an expert's weights the strides of a tensor map.
static bool valid_extent(int64_t row_blocks, int64_t m, int64_t n) {
  return row_blocks * ((n + TN / 2 - 1) / (TN / 2)) < ((int64_t)1 << 30) && m * n < ((int64_t)1 << 38);
}

static bool null_or_misaligned(const void* p) { return !p || !aligned16(p); }

}  // namespace ep

using namespace ep;

extern "C" int ep_expert_gemm(const uint16_t* x, int64_t rows, int64_t K, const uint16_t* w, int n_w, int64_t N,
                              int transpose_w, const int32_t* cu_seqlens, int n_slots, const int32_t* slot_order,
                              const int32_t* rep_expert, int n_rep, uint16_t* y, int32_t* dev_status,
                              cudaStream_t stream) {
  if (!valid_slots(rows, n_w, cu_seqlens, n_slots, n_rep) || !valid_width(K) || !valid_width(N)) return EP_ERR_ARG;
  if (!valid_extent(rows / TM + n_slots, K, N)) return EP_ERR_ARG;
  if (rows == 0 || n_slots == 0) return EP_OK;
  if (null_or_misaligned(x) || null_or_misaligned(w) || null_or_misaligned(y)) return EP_ERR_ARG;
  ExpertArgs a = {};
  a.rows = rows, a.N = (int)N, a.K = (int)K, a.n_slots = n_slots, a.n_w = n_w, a.n_rep = rep_expert ? n_rep : 0;
  a.cu = cu_seqlens, a.slots = slot_order, a.rep = rep_expert, a.y = y, a.dev_status = dev_status;
  CUtensorMap ma, mb;
  if (!transpose_w && few_rows(rows, n_slots, n_w)) {
    if (!map_rows(&ma, x, rows, (int)K, FEW) || !map_weights(&mb, w, n_w, (int)N, (int)K, 128)) return EP_ERR_CUDA;
    return launch_few<Y_NT>(ma, mb, a, stream);
  }
  if (!map_rows(&ma, x, rows, (int)K, TM / 2)) return EP_ERR_CUDA;
  if (transpose_w) {
    if (!map_weights(&mb, w, n_w, (int)K, (int)N, TK)) return EP_ERR_CUDA;
    return launch_experts<Y_NN>(ma, mb, a, stream);
  }
  if (!map_weights(&mb, w, n_w, (int)N, (int)K, TN / 2)) return EP_ERR_CUDA;
  return launch_experts<Y_NT>(ma, mb, a, stream);
}

extern "C" int ep_expert_up(const uint16_t* x, int64_t rows, int64_t H, const uint16_t* w, int n_w, int64_t I,
                            const int32_t* cu_seqlens, int n_slots, const int32_t* slot_order,
                            const int32_t* rep_expert, int n_rep, uint16_t* h, uint16_t* gu, int32_t* dev_status,
                            cudaStream_t stream) {
  if (!valid_slots(rows, n_w, cu_seqlens, n_slots, n_rep) || !valid_width(H) || !valid_width(I)) return EP_ERR_ARG;
  if (!valid_extent(rows / TM + n_slots, H, I)) return EP_ERR_ARG;
  if (rows == 0 || n_slots == 0) return EP_OK;
  if (null_or_misaligned(x) || null_or_misaligned(w) || null_or_misaligned(h) || !aligned16(gu)) return EP_ERR_ARG;
  ExpertArgs a = {};
  a.rows = rows, a.N = (int)I, a.K = (int)H, a.n_slots = n_slots, a.n_w = n_w, a.n_rep = rep_expert ? n_rep : 0;
  a.cu = cu_seqlens, a.slots = slot_order, a.rep = rep_expert, a.y = h, a.y2 = gu, a.dev_status = dev_status;
  CUtensorMap ma, mb;
  if (!map_weights(&mb, w, n_w, (int)(2 * I), (int)H, 128)) return EP_ERR_CUDA;
  if (few_rows(rows, n_slots, n_w)) {
    if (!map_rows(&ma, x, rows, (int)H, FEW)) return EP_ERR_CUDA;
    return launch_few<UP>(ma, mb, a, stream);
  }
  if (!map_rows(&ma, x, rows, (int)H, TM / 2)) return EP_ERR_CUDA;
  return launch_experts<UP>(ma, mb, a, stream);
}

extern "C" int ep_expert_up_backward(const uint16_t* dy, int64_t rows, int64_t H, const uint16_t* w2, int n_w,
                                     int64_t I, const uint16_t* gu, const int32_t* cu_seqlens, int n_slots,
                                     const int32_t* slot_order, const int32_t* rep_expert, int n_rep, uint16_t* dgu,
                                     uint16_t* h, int32_t* dev_status, cudaStream_t stream) {
  if (!valid_slots(rows, n_w, cu_seqlens, n_slots, n_rep) || !valid_width(H) || !valid_width(I)) return EP_ERR_ARG;
  if (!valid_extent(rows / TM + n_slots, H, I)) return EP_ERR_ARG;
  if (rows == 0 || n_slots == 0) return EP_OK;
  if (null_or_misaligned(dy) || null_or_misaligned(w2) || null_or_misaligned(gu) || null_or_misaligned(dgu) ||
      !aligned16(h))
    return EP_ERR_ARG;
  ExpertArgs a = {};
  a.rows = rows, a.N = (int)I, a.K = (int)H, a.n_slots = n_slots, a.n_w = n_w, a.n_rep = rep_expert ? n_rep : 0;
  a.cu = cu_seqlens, a.slots = slot_order, a.rep = rep_expert, a.y = dgu, a.y2 = h, a.gu = gu;
  a.dev_status = dev_status;
  CUtensorMap ma, mb;
  if (!map_rows(&ma, dy, rows, (int)H, TM / 2) || !map_weights(&mb, w2, n_w, (int)H, (int)I, TK)) return EP_ERR_CUDA;
  return launch_experts<UP_BACKWARD>(ma, mb, a, stream);
}

extern "C" int ep_expert_wgrad(const uint16_t* a_rows, const uint16_t* b_rows, int64_t rows, int64_t M, int64_t N,
                               const int32_t* cu_seqlens, int n_slots, const int32_t* slot_order, float* g_home,
                               int n_home, int64_t ld_home, void* g_rep, int rep_dtype, int n_rep, int64_t ld_rep,
                               int accumulate, int32_t* dev_status, cudaStream_t stream) {
  if (!valid_slots(rows, n_home, cu_seqlens, n_slots, n_rep) || !valid_width(M) || !valid_width(N)) return EP_ERR_ARG;
  if (rep_dtype != EP_DTYPE_F32 && rep_dtype != EP_DTYPE_BF16) return EP_ERR_ARG;
  if (!valid_extent((M + TM - 1) / TM * n_slots, M, N) || ld_home < M * N || ld_home % 4) return EP_ERR_ARG;
  if (g_rep && (!aligned16(g_rep) || ld_rep < M * N || ld_rep % (rep_dtype == EP_DTYPE_F32 ? 4 : 8))) return EP_ERR_ARG;
  if (n_slots == 0) return EP_OK;
  if (null_or_misaligned(g_home) || (rows > 0 && (null_or_misaligned(a_rows) || null_or_misaligned(b_rows))))
    return EP_ERR_ARG;
  ExpertArgs a = {};
  a.rows = rows, a.N = (int)N, a.K = (int)M, a.n_slots = n_slots, a.n_w = n_home, a.n_rep = g_rep ? n_rep : 0;
  a.cu = cu_seqlens, a.slots = slot_order, a.g_home = g_home, a.g_rep = g_rep, a.ld_home = ld_home, a.ld_rep = ld_rep;
  a.rep_bf16 = rep_dtype == EP_DTYPE_BF16, a.dev_status = dev_status;
  a.add_home = accumulate != 0, a.add_rep = accumulate != 0 && accumulate != EP_ACCUMULATE_HOME;
  CUtensorMap ma, mb;
  // without rows nothing is read, but a map needs an address
  if (!map_rows(&ma, rows ? (const void*)a_rows : g_home, rows ? rows : 1, (int)M, TK) ||
      !map_rows(&mb, rows ? (const void*)b_rows : g_home, rows ? rows : 1, (int)N, TK))
    return EP_ERR_CUDA;
  return launch_experts<WGRAD>(ma, mb, a, stream);
}
