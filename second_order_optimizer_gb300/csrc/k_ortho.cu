// Orthogonalised updates by Newton-Schulz products.  Of a matrix G with small side s and long
// side l (X stands for G or, by its columns, for G^T):
//   X_0 = G / (|G|_F + eps);   L = X X^T,  M = a I + b L + c L^2,  X <- M X   per step,
// after which the singular values of X are near one (a polynomial of each: a t + b t^3 + c t^5).
//
// Per step two symmetric products (s^2 l and s^3 multiply-adds over their distinct halves) and one
// whole one (s^2 l): bound by the tensor cores where there are tiles for every SM, by the chain of
// launches where there are not.
//
// All these matrices are polynomials of one L, so they commute, and steps can be taken on the small
// side alone: L' = M L M and P = M' M are symmetric products of size s, and X is read and written
// once per group of steps (X <- P X) instead of once per step.  With r = l / s a group of g steps
// costs s^3 (3 r + 4 g - 3) instead of s^3 g (3 r + 1): at l = 4 s, three and two steps together take
// 38 s^3 for 65.  What L was rounded by grows by max |M|^2 (11.9 for the default coefficients) with
// every step that it is not formed anew from X, so groups end before that passes 150: three
// steps.  X is rounded less often and L_0 is formed from X_0 itself, so the result is no less
// exact (emulated: 1.9e-3 to 3.6e-3 off where single steps are 1.9e-3 to 7e-3).
//
// Operands are fp16, not bf16: every matrix here is bounded (|X| <= u, |L| <= u^2, |M| <= v with u, v
// from the polynomial on [0, u]), so a power of two per matrix and step brings it to just below
// 2^15 and fp16's 11 bits serve where bf16 would give 8.  After five steps the result is 2e-3 to
// 3e-3 off in norm (1.7e-3 of it the rounding of a bf16 result); bf16 operands gave 1e-2 to 2e-2 in the
// same emulation.  X_0 is G times a power of two, exact for bf16; what is left of the norm, a
// factor r, enters the first step's products in fp32.  The full arithmetic (fp32 tensors) keeps
// each matrix as two fp16 values, v = hi + lo (22 bits), multiplies hi hi + hi lo + lo hi, and
// drains the accumulator every 64 k into fp32 registers (the tensor cores' sums round towards
// zero; every 128 k, the small products in between, were 6e-6 off): about 1e-6 off.
//
// One kernel serves all products: CTA pairs (tcgen05 cta_group::2) on 256 x 256 tiles of all the
// call's matrices, persistent, a warp for TMA, one for the MMAs, eight for the epilogue, two
// accumulators in TMEM so that a tile's epilogue runs beside the next one's products; single CTAs
// on 128 x 128 tiles where the larger ones would leave SMs idle.  A matrix
// is never transposed: the operand whose k runs down the rows of X is read as it lies, as an
// MN-major tile.  Of a symmetric product the tiles on and above the diagonal are computed; the
// epilogue stores each of them (through shared memory, by TMA) and its transpose.
#include "kfac_internal.cuh"
#include "per_device.h"
#include "ring.h"
#include "tc_prims.cuh"
#include "tensor_map.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <type_traits>
#include <utility>
#include <vector>

namespace kfac {
namespace ortho {

__device__ DevStatus g_status;   // device-side errors, read by kfac_operator_status

namespace {

constexpr int kMaxGroup = 24;        // matrices per launch of the norm
constexpr int kMaxSide = 32768;      // no accumulator sums more terms
constexpr int kMaxSteps = 32;
constexpr int kPrepThreads = 256;
constexpr int kPrepBlocks = 512;     // per matrix, at most

// ------------------------------------------------------------------------- norm and scaling

// One matrix of the call: x (step: the gradient g, with the momentum m).
struct PrepTask {
  const void* x;
  float* m;
  int64_t ldx, ldm;
  __half *hi, *lo;         // X_0, rows of `pitch`
  float* part;             // [blocks][3]: squares by range
  float* r;                // the factor r, the word of a lost product (see Task) and the exponent j
  int rows, cols, pitch;
  int tx;                  // threads per row (a power of two)
  int vec;                 // whole 16-byte vectors of x (and of m)
};
struct PrepLaunch {
  PrepTask task[kMaxGroup];
  int block_start[kMaxGroup + 1];
  int count;
  double eps;
  float mu;
  int nesterov;
};

__device__ __forceinline__ int task_of(const int* start, int count, int block) {
  int q = 0;
  while (q + 1 < count && block >= start[q + 1]) ++q;
  return q;
}

template <typename T, int N> struct alignas(N * sizeof(T)) Vec { T v[N]; };

// The pieces of n elements that a thread takes of a matrix: tx threads per row, rows apart by the
// matrix's blocks.
struct Pieces {
  int64_t row, row_step;
  int c, c0, c_step;
  __device__ __forceinline__ Pieces(const PrepTask& t, int n, int block, int blocks) {
    const int rpb = kPrepThreads / t.tx;
    row = (int64_t)block * rpb + threadIdx.x / t.tx;
    row_step = (int64_t)blocks * rpb;
    c = c0 = (int)(threadIdx.x % t.tx) * n;
    c_step = t.tx * n;
  }
  __device__ __forceinline__ bool next(const PrepTask& t, int64_t* r, int* col) {
    if (c >= t.cols) {
      c = c0;
      row += row_step;
    }
    if (row >= t.rows || c >= t.cols) return false;
    *r = row;
    *col = c;
    c += c_step;
    return true;
  }
};

// N values of the matrix to orthogonalise from column c of a row: x, or with the momentum
// m <- mu m + g the update g + mu m (nesterov) or m.  Loading and using them are apart, so that
// several pieces' loads are in flight.
template <typename T, int N, bool kStep> struct Piece {
  static constexpr int F = N < 4 ? N : 4;
  Vec<T, N> g;
  Vec<float, F> m[kStep ? N / F : 1];
  __device__ __forceinline__ void load(const PrepTask& t, int64_t row, int c) {
    g = *reinterpret_cast<const Vec<T, N>*>(static_cast<const T*>(t.x) + row * t.ldx + c);
    if constexpr (kStep) {
#pragma unroll
      for (int j = 0; j < N / F; ++j)
        m[j] = *reinterpret_cast<const Vec<float, F>*>(t.m + row * t.ldm + c + j * F);
    }
  }
  // kFresh: m is still the one before this step; it is updated and written.
  template <bool kFresh>
  __device__ __forceinline__ void use(float mu, int nesterov, const PrepTask& t, int64_t row, int c,
                                      float (&u)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = to_f32<T>(g.v[i]);
    if constexpr (kStep) {
#pragma unroll
      for (int j = 0; j < N / F; ++j) {
        if (kFresh) {
#pragma unroll
          for (int i = 0; i < F; ++i) m[j].v[i] = fmaf(mu, m[j].v[i], u[j * F + i]);
          *reinterpret_cast<Vec<float, F>*>(t.m + row * t.ldm + c + j * F) = m[j];
        }
#pragma unroll
        for (int i = 0; i < F; ++i)
          u[j * F + i] = nesterov ? fmaf(mu, m[j].v[i], u[j * F + i]) : m[j].v[i];
      }
    }
  }
};
// f(row, column, values) for every piece of a thread.
template <typename T, int N, bool kStep, bool kFresh, typename F>
__device__ __forceinline__ void each_piece(const PrepLaunch& l, const PrepTask& t, int block, int blocks, F f) {
  constexpr int AHEAD = 4;
  Pieces walk(t, N, block, blocks);
  for (bool more = true; more;) {
    Piece<T, N, kStep> p[AHEAD];
    int64_t row[AHEAD];
    int c[AHEAD];
    bool ok[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      ok[k] = walk.next(t, &row[k], &c[k]);
      if (ok[k]) p[k].load(t, row[k], c[k]);
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (!ok[k]) continue;
      float u[N];
      p[k].template use<kFresh>(l.mu, l.nesterov, t, row[k], c[k], u);
      f(row[k], c[k], u);
    }
    more = ok[AHEAD - 1];
  }
}

// A thread's squares: plainly, unless its largest value says that they overflow or vanish; then of
// the values times 2^-84 (from 2^40 on: 2^30 squares below 2^128) or 2^88 (below 2^-30, down to
// 2^-149), in a second round.  A value so small that its square vanishes beside a larger one is
// not missed.
struct Squares {
  float mid = 0.f, top = 0.f, scaled = 0.f;
  template <int N> __device__ __forceinline__ void add(const float (&u)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      mid = fmaf(u[i], u[i], mid);
      top = fmaxf(top, fabsf(u[i]));
    }
  }
  __device__ __forceinline__ bool big() const { return top >= 0x1p40f; }
  __device__ __forceinline__ bool unsafe() const {   // (a NaN is in mid)
    return big() || (top < 0x1p-30f && top > 0.f && mid == mid);
  }
  template <int N> __device__ __forceinline__ void add_scaled(const float (&u)[N]) {
    const float by = big() ? 0x1p-84f : 0x1p88f;
#pragma unroll
    for (int i = 0; i < N; ++i) scaled = fmaf(u[i] * by, u[i] * by, scaled);
  }
  // scale_factors' three sums
  __device__ __forceinline__ void finish(float (&sums)[3]) const {
    sums[0] = big() ? scaled : 0.f;
    sums[1] = unsafe() && mid == mid ? 0.f : mid;
    sums[2] = unsafe() && !big() ? scaled : 0.f;
  }
};
template <typename T, int N, bool kStep>
__device__ __forceinline__ void sum_squares(const PrepLaunch& l, const PrepTask& t, int block, int blocks,
                                            float (&sums)[3]) {
  Squares s;
  each_piece<T, N, kStep, true>(l, t, block, blocks, [&](int64_t, int, const float (&u)[N]) { s.add(u); });
  if (s.unsafe())
    each_piece<T, N, kStep, false>(l, t, block, blocks,
                                   [&](int64_t, int, const float (&u)[N]) { s.add_scaled(u); });
  s.finish(sums);
}

template <typename T, bool kStep>
__global__ void __launch_bounds__(kPrepThreads) ortho_norm_kernel(const __grid_constant__ PrepLaunch g) {
  __shared__ float red[3][kPrepThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int q = task_of(g.block_start, g.count, blockIdx.x);
  const PrepTask& t = g.task[q];
  const int block = blockIdx.x - g.block_start[q], blocks = g.block_start[q + 1] - g.block_start[q];
  float v[3];
  if (t.vec) sum_squares<T, 16 / (int)sizeof(T), kStep>(g, t, block, blocks, v);
  else sum_squares<T, 1, kStep>(g, t, block, blocks, v);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (threadIdx.x % 32 == 0) red[k][threadIdx.x / 32] = v[k];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    float sum = 0.f;
    for (int w = 0; w < kPrepThreads / 32; ++w) sum += red[threadIdx.x][w];
    t.part[block * 3 + threadIdx.x] = sum;
  }
}

// From the squares by range (big, plain, small): 2^k (in two factors, each within fp32's range)
// with |x 2^k|_F in [2^13, 2^14), and r and j with x / (|x| + eps) = r 2^-j x 2^k, where 2^-j is the power
// of two from |x| / (|x| + eps) up.  (j is 0 unless |x| < eps.  Then all of X is that small, and is kept
// times a power of two through the steps, see Plan: scaled as if |X| were 1 it would fall out of fp16's
// range.  Of 256 x 512 in full arithmetic, |x| = 1e-13 and eps = 1e-7 were 4.7e-4 off, 1e-15 4.7e-2.)
__device__ __forceinline__ void scale_factors(const double (&sums)[3], double eps, float (&up)[2], float* r_out,
                                              float* j_out) {
  const double x = sqrt(sums[0] * 0x1p168 + sums[1] + sums[2] * 0x1p-176), norm = x + eps;
  float r = 0.f;
  int k = 0, j = 0;
  if (x > 0.0 && isfinite(norm)) {
    // by the bits of the doubles (both normal): 64-bit functions are slow, and all wait for this thread
    const long long xb = __double_as_longlong(x), nb = __double_as_longlong(norm);
    k = 14 - ((int)(xb >> 52) - 1022);       // x < 2^(14 - k)
    j = (int)((nb - xb) >> 52);              // x / norm <= 2^-j < 2 x / norm
    r = (float)(__longlong_as_double((long long)(1023 + j - k) << 52) / norm);
  } else if (x != 0.0) {                     // Inf and NaN reach everything through r
    r = __int_as_float(0x7fffffff);
  }
  const int k0 = min(max(k, -126), 126);
  up[0] = __int_as_float((127 + k0) << 23);
  up[1] = __int_as_float((127 + k - k0) << 23);
  *r_out = r;
  *j_out = (float)j;
}

template <typename T, bool kStep, bool kFull>
__global__ void __launch_bounds__(kPrepThreads) ortho_scale_kernel(const __grid_constant__ PrepLaunch g) {
  __shared__ double sums[3];
  __shared__ float factor[2];
  pdl_wait();
  pdl_trigger();
  const int q = task_of(g.block_start, g.count, blockIdx.x);
  const PrepTask& t = g.task[q];
  const int block = blockIdx.x - g.block_start[q], blocks = g.block_start[q + 1] - g.block_start[q];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp < 3) {   // the same order in every block
    double sum = 0.0;
    for (int b = lane; b < blocks; b += 32) sum += (double)t.part[b * 3 + warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sums[warp] = sum;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const double all[3] = {sums[0], sums[1], sums[2]};
    float up[2], r, j;
    scale_factors(all, g.eps, up, &r, &j);
    factor[0] = up[0];
    factor[1] = up[1];
    if (block == 0) {
      t.r[0] = r;
      t.r[1] = 0.f;
      t.r[2] = j;
    }
  }
  __syncthreads();
  const float up0 = factor[0], up1 = factor[1];
  auto store = [&](int64_t row, int c, auto& u) {
    constexpr int n = sizeof(u) / sizeof(float);
    Vec<__half, n> h, l;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float v = u[i] * up0 * up1;
      h.v[i] = __float2half_rn(v);
      if (kFull) l.v[i] = __float2half_rn(v - __half2float(h.v[i]));
    }
    *reinterpret_cast<Vec<__half, n>*>(t.hi + row * t.pitch + c) = h;
    if (kFull) *reinterpret_cast<Vec<__half, n>*>(t.lo + row * t.pitch + c) = l;
  };
  if (t.vec) each_piece<T, 16 / (int)sizeof(T), kStep, false>(g, t, block, blocks, store);
  else each_piece<T, 1, kStep, false>(g, t, block, blocks, store);
}

// -------------------------------------------------------------------------------- products

// What becomes of a product: another matrix of the iteration, or with the last X the direction or
// the weights.
enum { TO_MATRIX, TO_OUT, TO_WEIGHTS };

// out = alpha r^rpow 2^e A B^T [+ beta add + diag I], stored as fp16, or as it is below.  X before step k
// is kept times 2^max(0, j + shift_k): of the product of an X, e takes that away (xpow times), and adds
// what the X that it gives has.
struct Task {
  int64_t out_ld;
  void* out;                    // TO_OUT: the direction; TO_WEIGHTS: the weights, fp32
  const __half *add_hi, *add_lo;   // or null
  __half *mirror_hi, *mirror_lo;   // upper: the result itself, whose other half is stored directly
  float* r;                     // r; a word that is not 0 once a product of this matrix is lost (a wait gave
                                // up, its tile was not stored: the last launch makes the matrix NaN, or
                                // leaves its weights); j
  float alpha, beta, diag;
  float keep, rate;             // TO_WEIGHTS: W <- keep W - rate X
  int rpow, xpow, shift_in, shift_out, add_pitch, mirror_pitch;
  int M, N, kblocks;            // sizes of the product; k in blocks of 64
  int tiles_m, upper;           // upper: symmetric, tiles on and above the diagonal
  int mn_a, mn_b;               // operands read as MN-major tiles
  int same_ab;                  // A is B
};
enum { MAP_A, MAP_B, MAP_STORE, MAPS };   // operands and result
template <bool kFull> struct Launch {
  static constexpr int TASKS = kFull ? 24 : 48;   // a kernel's parameters end at 32764 bytes
  int give_up;             // self-test: a warp's wait for the first tile is taken for one that ran out
  CUtensorMap maps[TASKS][MAPS * (kFull ? 2 : 1)];
  Task task[TASKS];
  int tile_start[TASKS + 1];
  int count;
};

template <bool kFull, bool kPair> struct Cfg {
  static constexpr int TILE = kPair ? 256 : 128;
  static constexpr int BK = 64;
  static constexpr int HALF = 128 * BK * 2;              // 128 rows (or features) of an operand
  static constexpr int STAGE = HALF * 2 * (kFull ? 2 : 1);
  static constexpr int STAGES = kFull ? 3 : 5;
  static constexpr int NBUF = kFull ? 1 : 2;             // 16 KB store buffers per epilogue group
  static constexpr int BUF = 128 * 64 * 2;
  static constexpr int SUB = kFull ? 1 : 1 << 20;        // k blocks per drain
  static constexpr int CW = TILE / 2;                    // columns of an epilogue warp
  static constexpr int TMEM = 2 * TILE;
  // warps 0 and 1: TMA, MMA; 4 to 11: epilogue (whole warpgroups, for the register split below)
  static constexpr int EPI0 = 4, EPI_WARPS = 8, THREADS = 32 * (EPI0 + EPI_WARPS);
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE + 2 * NBUF * BUF + 512;
  static_assert(SMEM <= 232448, "fits the per-CTA shared memory");
};
// Full arithmetic on pairs keeps 128 running sums a thread.  384 threads are launched with at most
// 168 registers each, 64512; the epilogue's 256 take 232 and leave the others 40.
constexpr int kLaunchRegs = 168, kEpilogueRegs = 232, kOtherRegs = 40;
static_assert(sizeof(Launch<true>) <= 32764 && sizeof(Launch<false>) <= 32764 &&
              Launch<true>::TASKS <= 2 * kMaxGroup && Launch<false>::TASKS <= 2 * kMaxGroup, "one launch");
static_assert(256 * kEpilogueRegs + 128 * kOtherRegs <= 384 * kLaunchRegs, "register split");

__device__ __forceinline__ void umma_pair_by(uint32_t leader, uint32_t d, uint64_t a, uint64_t b,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit_pair_by(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n"
      " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;\n}\n" ::"r"(tc::smem_u32(bar)),
      "h"((uint16_t)3), "r"(leader)
      : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
constexpr long long kLandCycles = 1 << 20;   // 0.5 ms: of copies and products in flight
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y,
                                            int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(tc::smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void group_sync(int id) {   // the 128 threads of an epilogue group
  asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}

// Whether all 128 say yes.
__device__ __forceinline__ bool group_all(int id, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.and.pred q, %2, 128, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(all)
      : "r"((uint32_t)ok), "r"(id)
      : "memory");
  return all != 0;
}

// Tile t of the launch: its task, row and column block.
template <bool kFull>
__device__ __forceinline__ void tile_of(const Launch<kFull>& g, int t, int* q, int* ti, int* tj) {
  int p = 0;
  while (p + 1 < g.count && t >= g.tile_start[p + 1]) ++p;
  t -= g.tile_start[p];
  *q = p;
  if (g.task[p].upper) {   // column block j holds j + 1 tiles
    int j = (int)((sqrtf(8.f * (float)t + 1.f) - 1.f) * 0.5f);
    while (j * (j + 1) / 2 > t) --j;
    while ((j + 1) * (j + 2) / 2 <= t) ++j;
    *tj = j;
    *ti = t - j * (j + 1) / 2;
  } else {
    *ti = t % g.task[p].tiles_m;
    *tj = t / g.task[p].tiles_m;
  }
}

// Two fp16 roundings in a word; the first at the lower address.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// The epilogue's store buffers: 64 columns of the CTA's 128 rows, in the 128-byte swizzle of the
// store maps.  w: this thread's row, word j of columns 2 j, 2 j + 1.
__device__ __forceinline__ void put_rows(uint8_t* buf, int row, const uint32_t (&w)[32]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4*>(buf + row * 128 + ((j ^ (row & 7)) << 4)) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}
// The same transposed, straight to memory: row c of the other half of the symmetric matrix gets
// this tile's column c.  Neighbouring lanes trade values so that each writes whole words of
// columns c and c + 1, 64 bytes of each per warp.  (By way of shared memory and TMA, as above, it
// took part of the bandwidth that the operands need: 13 to 14 us a tile of 2048 k against 11.5.)
// out: at row c0, column of this thread's row rounded down to even; cols: columns that exist.
__device__ __forceinline__ void put_columns(__half* out, int64_t pitch, bool row_ok, int cols,
                                            const uint32_t (&w)[32]) {
  const bool odd = threadIdx.x & 1;
  out += odd ? pitch : 0;
  const int mine = row_ok ? cols - (odd ? 1 : 0) : 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {   // columns 2 j, 2 j + 1
    const uint32_t o = __shfl_xor_sync(0xffffffffu, w[j], 1);
    const uint32_t word = odd ? __byte_perm(w[j], o, 0x3276) : __byte_perm(w[j], o, 0x5410);
    if (2 * j < mine) *reinterpret_cast<uint32_t*>(out + 2 * j * pitch) = word;
  }
}

// A block on the diagonal of a product of two different matrices: the elements on and above it as
// they are, those above it transposed, so that the matrix is symmetric to the last bit.  (Rounding
// leaves the product of two matrices that commute a little unsymmetric, and of that part the
// polynomial's next step sees b L without c L^2, which for the symmetric part takes most of it
// back: three steps on the small side, then three more, were 1.2e-2 off where 2e-3 is due.  A matrix times
// itself is symmetric in half arithmetic as it comes; in full arithmetic up to its last bits, since hi lo
// and lo hi are added in another order on the two sides.  Stored by one half too, results of 3 to 12
// steps agreed to three digits, and 129 x 512 took 195 us for 140.)  to: row gr (its column c0);
// mirror: row c0, column gr rounded down to even.
__device__ __forceinline__ void put_diagonal(__half* to, __half* mirror, int64_t pitch, int gr, int c0, int n,
                                             const uint32_t (&w)[32]) {
  if (gr < n) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + 8 * j;
      if (c >= gr) {       // (columns from n to the pitch take whatever there is)
        *reinterpret_cast<uint4*>(to + 8 * j) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
      } else if (c + 8 > gr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const __half2 h = *reinterpret_cast<const __half2*>(&w[4 * j + i / 2]);
          if (c + i >= gr) to[8 * j + i] = i & 1 ? h.y : h.x;
        }
      }
    }
  }
  const bool odd = gr & 1;
  const int e = gr & ~1;   // this lane's words hold rows e and e + 1
#pragma unroll
  for (int j = 0; j < 32; ++j) {   // columns 2 j, 2 j + 1
    const uint32_t o = __shfl_xor_sync(0xffffffffu, w[j], 1);
    const uint32_t word = odd ? __byte_perm(w[j], o, 0x3276) : __byte_perm(w[j], o, 0x5410);
    const int k = 2 * j + odd, c = c0 + k;
    __half* at = mirror + (int64_t)k * pitch;
    if (c < n && c > e + 1) *reinterpret_cast<uint32_t*>(at) = word;
    else if (c < n && c == e + 1) *at = __ushort_as_half((unsigned short)(word & 0xffffu));
  }
}

template <int TO, typename T, bool kFull, bool kPair>
__global__ void __launch_bounds__(Cfg<kFull, kPair>::THREADS, 1)
    ortho_product_kernel(const __grid_constant__ Launch<kFull> g) {
  using C = Cfg<kFull, kPair>;
  constexpr int STAGES = C::STAGES, TILE = C::TILE, CTAS = kPair ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* bufs = smem + (size_t)STAGES * C::STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(bufs + 2 * C::NBUF * C::BUF);
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drained = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* copies = tmem_slot + 2;   // loads of operands that the producer has issued
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int total = g.tile_start[g.count];
  const uint32_t rank = kPair ? tc::cluster_rank() : 0;
  const int unit = (int)(blockIdx.x / CTAS), units = (int)(gridDim.x / CTAS);
  // a role that gives up stops the peer CTA's roles too
  const uint32_t peer_abort = kPair ? tc::mapa((const void*)abort_flag, rank ^ 1u) : 0;
  auto give_up = [&](int info) {
    report_error(&g_status, KFAC_ERR_TIMEOUT, -1, info);
    *abort_flag = 1;
    if (kPair) tc::st_cluster_u32(peer_abort, 1u);
  };
  auto block_sync = [&]() {
    if constexpr (kPair) tc::cluster_sync();
    else __syncthreads();
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&acc_full[b], 1);
      tc::mbar_init(&acc_empty[b], CTAS * C::EPI_WARPS);
    }
    tc::mbar_init(drained, 1);
    *abort_flag = 0;
    *copies = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tc::tmem_alloc_pair(tmem_slot, C::TMEM);
      tc::tmem_relinquish_pair();
    } else {
      tc::tmem_alloc(tmem_slot, C::TMEM);
      tc::tmem_relinquish();
    }
  }
  if (warp == 0 && unit < total) {   // the first tile's maps, before anything waits
    int q, ti, tj;
    tile_of(g, unit, &q, &ti, &tj);
    if (lane < MAPS) tc::tma_prefetch_desc(&g.maps[q][lane]);
  }
  tc::tc_fence_before();
  __syncwarp();
  block_sync();   // the barriers initialised and TMEM allocated (of both CTAs)
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  // a diagonal tile of a matrix with itself: this CTA's rows of A are its rows of B
  auto shared_ab = [&](const Task& k, int ti, int tj) { return k.same_ab && ti == tj; };

  if (warp < C::EPI0) {
    if constexpr (kFull && kPair) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------------- TMA producer
      const uint32_t full0 = kPair ? tc::mapa(full, 0) : 0;   // the even CTA's stage barriers
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        int q, ti, tj;
        tile_of(g, t, &q, &ti, &tj);
        const Task& k = g.task[q];
        const bool ab = shared_ab(k, ti, tj);
        const int arow = ti * TILE + (int)rank * 128, brow = tj * TILE + (int)rank * 128;
        const int mn_a = k.mn_a, mn_b = k.mn_b, kblocks = k.kblocks;
        const CUtensorMap* maps = g.maps[q];
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!tc::mbar_wait(&empty[stage], phase ^ 1, abort_flag)) {
            give_up(41);
            ok = false;
            break;
          }
          const uint32_t fb = full0 + (uint32_t)(stage * sizeof(uint64_t));
          if (rank == 0)
            tc::mbar_expect_tx(&full[stage], CTAS * (ab ? C::STAGE / 2 : C::STAGE));   // (both CTAs' loads)
          uint8_t* at = smem + (size_t)stage * C::STAGE;
          auto load = [&](uint8_t* dst, const CUtensorMap* m, int mn, int row) {
            if constexpr (kPair) {
              if (mn) tc::tma_load_3d_pair(dst, m, fb, 0, kb * C::BK, row / 64);
              else tc::tma_load_2d_pair(dst, m, fb, kb * C::BK, row);
            } else {
              if (mn) tma_load_3d(dst, m, &full[stage], 0, kb * C::BK, row / 64);
              else tc::tma_load_2d(dst, m, &full[stage], kb * C::BK, row);
            }
          };
#pragma unroll
          for (int part = 0; part < (kFull ? 2 : 1); ++part) {
            if (!ab) load(at + part * 2 * C::HALF, maps + MAP_A + part * MAPS, mn_a, arow);
            load(at + part * 2 * C::HALF + C::HALF, maps + MAP_B + part * MAPS, mn_b, brow);
          }
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      *copies = (uint32_t)issued;
    } else if (warp == 1 && rank == 0) {
      // ---------------------------------------------------------------- MMA issuer
      const uint32_t leader = tc::elect_leader();
      auto mma = [&](uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
        if constexpr (kPair) umma_pair_by(leader, d, a, b, idesc, accumulate);
        else tc::umma_f16_by(leader, d, a, b, idesc, accumulate);
      };
      auto commit = [&](uint64_t* bar) {
        if constexpr (kPair) commit_pair_by(leader, bar);
        else tc::umma_commit_by(leader, bar);
      };
      int stage = 0, gsub = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        int q, ti, tj;
        tile_of(g, t, &q, &ti, &tj);
        const bool ab = shared_ab(g.task[q], ti, tj);
        const int kblocks = g.task[q].kblocks, mn_a = g.task[q].mn_a, mn_b = g.task[q].mn_b;
        const uint32_t idesc = tc::make_idesc(0, TILE, TILE) | (mn_a ? tc::kIdescMnA : 0) |
                               (mn_b ? tc::kIdescMnB : 0);
        // per 16 k: 32 bytes along a K-major row, two groups of 8 rows down an MN-major tile
        const uint64_t step_a = mn_a ? 2048 >> 4 : 32 >> 4, step_b = mn_b ? 2048 >> 4 : 32 >> 4;
        auto desc = [&](uint32_t addr, int mn) {
          return mn ? tc::sdesc_mnmajor_sw128(addr, C::BK * 128) : tc::sdesc_kmajor_sw128(addr);
        };
        for (int kb0 = 0; kb0 < kblocks && ok; kb0 += C::SUB, ++gsub) {
          const int buf = gsub & 1, use = gsub >> 1;
          if (!tc::mbar_wait(&acc_empty[buf], (use & 1) ^ 1, abort_flag)) {
            if (leader) give_up(42);
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const uint32_t d = tmem + (uint32_t)(buf * TILE);
          const int kb1 = min(kblocks, kb0 + C::SUB);
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!tc::mbar_wait(&full[stage], phase, abort_flag)) {
              if (leader) give_up(43);
              ok = false;
              break;
            }
            tc::tc_fence_after();
            const uint32_t at = tc::smem_u32(smem + (size_t)stage * C::STAGE);
            const uint64_t a = desc(at + (ab ? C::HALF : 0), mn_a), b = desc(at + C::HALF, mn_b);
            constexpr uint64_t LO = 2 * C::HALF >> 4;   // from an operand's hi tile to its lo tile
            if constexpr (kFull) {   // the small terms first: fewer roundings at the sum's size
#pragma unroll
              for (int kk = 0; kk < C::BK / 16; ++kk) {
                const uint64_t ak = a + kk * step_a, bk = b + kk * step_b;
                mma(d, ak, bk + LO, idesc, kb > kb0 || kk > 0);
                mma(d, ak + LO, bk, idesc, 1u);
              }
            }
#pragma unroll
            for (int kk = 0; kk < C::BK / 16; ++kk)
              mma(d, a + kk * step_a, b + kk * step_b, idesc, kFull || kb > kb0 || kk > 0);
            commit(&empty[stage]);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (ok) commit(&acc_full[buf]);
        }
      }
    }
  } else {
    // -------------------------------------------------------------------- epilogue
    if constexpr (kFull && kPair) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
    constexpr int CW = C::CW;
    const int qd = warp & 3;                 // TMEM lane quarter this warp may access
    const int h = (warp - C::EPI0) >> 2;     // columns [CW h, CW h + CW) of the tile
    const int row = 32 * qd + lane;
    const bool issuer = qd == 0 && lane == 0;
    uint8_t* mybufs = bufs + h * C::NBUF * C::BUF;
    const uint32_t acc_empty0 = kPair ? tc::mapa(acc_empty, 0) : 0;
    auto release = [&](int buf) {   // this warp has read the accumulator
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kPair) tc::mbar_arrive_remote(acc_empty0 + (uint32_t)(buf * sizeof(uint64_t)));
        else tc::mbar_arrive(&acc_empty[buf]);
      }
    };
    int gsub = 0, turn = 0;
    bool ok = true;
    for (int t = unit; t < total; t += units) {
      int q, ti, tj;
      tile_of(g, t, &q, &ti, &tj);
      const Task& k = g.task[q];
      const bool quit = g.give_up && t == 0 && rank == 0 && warp == C::EPI0;
      const int kM = k.M, kN = k.N;
      const int r0 = ti * TILE + (int)rank * 128, gr = r0 + row;
      const int cols0 = tj * TILE + h * CW;
      const uint32_t lane_tmem = tmem + ((uint32_t)(32 * qd) << 16) + (uint32_t)(h * CW);
      // TO_WEIGHTS: 32 rows x 32 columns of W, loaded ahead of their use
      float w_old[TO == TO_WEIGHTS ? 32 : 1];
      auto load_weights = [&](int c0) {
        if constexpr (TO == TO_WEIGHTS) {
          const float* from = static_cast<const float*>(k.out) + (int64_t)(r0 + 32 * qd) * k.out_ld + c0 + lane;
          const int rows = min(32, kM - (r0 + 32 * qd));
#pragma unroll
          for (int i = 0; i < 32; ++i)
            w_old[i] = i < rows && c0 + lane < kN ? from[(int64_t)i * k.out_ld] : 0.f;
        }
      };
      load_weights(cols0);
      // 64 columns of this thread's row of the matrix to add, likewise
      // (full arithmetic has no registers to spare: there it is loaded when it is added)
      uint4 add[TO == TO_MATRIX ? 8 : 1];
      auto load_addend = [&](const __half* from, int c0) {
        if constexpr (TO == TO_MATRIX) {
          const uint4* at = reinterpret_cast<const uint4*>(from + (int64_t)gr * k.add_pitch + c0);
#pragma unroll
          for (int j = 0; j < 8; ++j) add[j] = gr < kM && c0 < kN ? at[j] : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      if (TO == TO_MATRIX && !kFull && k.add_hi) load_addend(k.add_hi, cols0);
      float alpha = k.alpha;
      if (k.xpow) {
        const float r = __ldg(k.r);
        const int j = (int)__ldg(k.r + 2);
        if (k.rpow) alpha *= k.rpow == 2 ? r * r : r;
        if (j > 0) alpha = ldexpf(alpha, max(0, j + k.shift_out) - k.xpow * max(0, j + k.shift_in));
      }
      float sum[kFull ? CW : 1];
      if constexpr (kFull) {
#pragma unroll
        for (int i = 0; i < CW; ++i) sum[i] = 0.f;
        const int nsub = (k.kblocks + C::SUB - 1) / C::SUB;
        for (int sub = 0; sub < nsub && ok; ++sub, ++gsub) {
          const int buf = gsub & 1, use = gsub >> 1;
          if (quit || !tc::mbar_wait(&acc_full[buf], use & 1, abort_flag)) {
            if (lane == 0) give_up(44);
            ok = false;
            break;
          }
          tc::tc_fence_after();
#pragma unroll
          for (int c = 0; c < CW / 32; ++c) {
            float v[32];
            tc::tmem_ld32(lane_tmem + (uint32_t)(buf * TILE + c * 32), v);
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[c * 32 + i] += v[i];
          }
          release(buf);
        }
      } else if (ok) {
        if (quit || !tc::mbar_wait(&acc_full[gsub & 1], (gsub >> 1) & 1, abort_flag)) {
          if (lane == 0) give_up(45);
          ok = false;
        }
        tc::tc_fence_after();
      }
      // One warp may see the abort flag where another, a moment later, finds its products done: what
      // stores by groups decides by groups, or some would wait in group_sync for ever.
      __syncwarp();
      ok = TO == TO_MATRIX ? group_all(1 + h, ok) : __all_sync(0xffffffffu, ok);
      if (!ok && TO == TO_MATRIX && issuer) {
        for (int u = t; u < total; u += units) {
          tile_of(g, u, &q, &ti, &tj);
          g.task[q].r[1] = 1.f;
        }
      }
      if (!ok && TO != TO_OUT) break;        // TO_OUT: the tiles from here on become NaN
      const bool lost = TO != TO_MATRIX && __ldcg(k.r + 1) != 0.f;
      if (TO == TO_OUT && lost) alpha = __int_as_float(0x7fffffff);
#pragma unroll
      for (int ch = 0; ch < CW / 64; ++ch) {       // 64 columns at a time
        const int c0 = cols0 + ch * 64;
        float v[64];
        if constexpr (kFull) {
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i] = sum[ch * 64 + i] * alpha;
        } else {
          if (ok) {
            uint32_t w0[32], w1[32];
            const uint32_t at = lane_tmem + (uint32_t)((gsub & 1) * TILE + ch * 64);
            tc::tmem_ld32_issue(at, w0);
            tc::tmem_ld32_issue(at + 32, w1);
            tc::tmem_ld_wait();
            tc::tmem_ld_use(w0);
            tc::tmem_ld_use(w1);
            if (ch == CW / 64 - 1) release(gsub & 1);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              v[i] = __uint_as_float(w0[i]) * alpha;
              v[32 + i] = __uint_as_float(w1[i]) * alpha;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) v[i] = 0.f;
          }
        }
        if (c0 >= kN || r0 >= kM) continue;   // (the whole group)
        if constexpr (TO != TO_MATRIX) {
          // 32 rows x 32 columns of the warp through shared memory, so that rows are written whole
          float* mine = reinterpret_cast<float*>(mybufs) + qd * 1024;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float4*>(mine + lane * 32 + ((j ^ (lane & 7)) << 2)) =
                  make_float4(v[half * 32 + 4 * j], v[half * 32 + 4 * j + 1], v[half * 32 + 4 * j + 2],
                              v[half * 32 + 4 * j + 3]);
            __syncwarp();
            const int c = c0 + half * 32 + lane;
            const int rows = TO == TO_WEIGHTS && lost ? 0 : min(32, kM - (r0 + 32 * qd));
            T* out = static_cast<T*>(k.out) + (int64_t)(r0 + 32 * qd) * k.out_ld + c;
            if (c < kN) {
              const int64_t ld = k.out_ld;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                if (i < rows) {
                  float x = mine[i * 32 + (((lane >> 2) ^ (i & 7)) << 2) + (lane & 3)];
                  if constexpr (TO == TO_WEIGHTS) x = fmaf(-k.rate, x, k.keep * w_old[i]);
                  else if (!ok) x = __int_as_float(0x7fffffff);
                  out[(int64_t)i * ld] = (T)x;
                }
              }
            }
            if (ch * 2 + half + 1 < CW / 32) load_weights(c0 + half * 32 + 32);
          }
        } else {
          if (k.add_hi) {
            const float beta = k.beta;
#pragma unroll
            for (int p = 0; p < (kFull ? 2 : 1); ++p) {
              if (kFull) load_addend(p ? k.add_lo : k.add_hi, c0);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const uint32_t e[4] = {add[j].x, add[j].y, add[j].z, add[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 f = unpack2(e[i]);
                  v[8 * j + 2 * i] = fmaf(beta, f.x, v[8 * j + 2 * i]);
                  v[8 * j + 2 * i + 1] = fmaf(beta, f.y, v[8 * j + 2 * i + 1]);
                }
              }
            }
            if (!kFull && ch + 1 < CW / 64) load_addend(k.add_hi, c0 + 64);
          }
          if (ti == tj) {   // (diag is 0 where there is no identity to add)
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (c0 + i == gr) v[i] += k.diag;
          }
          // hi (and lo) values, each as they are and, above the diagonal, transposed.  What lies above
          // goes by blocks of 128 whatever the tile is: a pair's diagonal tile has one above the
          // diagonal (1), one below it (-1) and two on it (0).
          const int side = !k.upper ? 2 : ti != tj ? 1 : kPair ? h - (int)rank : 0;
          uint32_t w[32];
#pragma unroll
          for (int part = 0; part < (kFull ? 2 : 1); ++part) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (kFull && part == 1) {
                const float2 hi = unpack2(w[i]);
                w[i] = pack2(v[2 * i] - hi.x, v[2 * i + 1] - hi.y);
              } else {
                w[i] = pack2(v[2 * i], v[2 * i + 1]);
              }
            }
            __half* const other = k.upper ? (part ? k.mirror_lo : k.mirror_hi) : nullptr;
            const int64_t pitch = k.mirror_pitch;
            if (side < 0) continue;
            if (side == 0 && !k.same_ab) {
              if (c0 + 64 > r0 + 32 * qd)   // (all of the warp's are below it otherwise)
                put_diagonal(other + gr * pitch + c0, other + c0 * pitch + (gr & ~1), pitch, gr, c0, kN, w);
              continue;
            }
            uint8_t* buf = mybufs + (turn % C::NBUF) * C::BUF;
            ++turn;
            if (issuer) bulk_wait_read<C::NBUF - 1>();   // the buffer's last store has read it
            group_sync(1 + h);
            put_rows(buf, row, w);
            tc::fence_proxy_async();
            group_sync(1 + h);
            if (issuer) {
              tma_store_2d(&g.maps[q][part * MAPS + MAP_STORE], buf, c0, r0);
              bulk_commit();
            }
            if (side == 1) put_columns(other + c0 * pitch + (gr & ~1), pitch, gr < kM, min(64, kN - c0), w);
          }
        }
      }
      if constexpr (!kFull) ++gsub;
    }
    if (issuer) bulk_wait();   // written before the next launch reads
  }
  tc::tc_fence_before();
  __syncwarp();
  block_sync();   // every MMA has completed; no peer arrival is pending
  if (*abort_flag) {   // (both CTAs' are set)
    // A role gave up, whichever and whenever: memory goes only after the copies have landed and the products
    // have ended.  Both CTAs' complete on the even one's barriers; where one CTA has issued more copies
    // than the other a barrier does not turn, and the limit outlasts them.
    volatile int never = 0;
    if (rank == 0 && threadIdx.x == 0) {
      const int issued = (int)(kPair ? max(*copies, ld_cluster_u32(tc::mapa(copies, 1))) : *copies);
      for (int s = 0; s < STAGES; ++s)
        if (const int uses = ring_uses(issued, s, STAGES))
          tc::mbar_wait(&full[s], ring_last_parity(uses), &never, kLandCycles);
    }
    if (rank == 0 && warp == 1) {
      const uint32_t leader = tc::elect_leader();   // the lane that issued them
      if constexpr (kPair) commit_pair_by(leader, drained);
      else tc::umma_commit_by(leader, drained);
      tc::mbar_wait(drained, 0, &never, kLandCycles);
    }
    __syncwarp();
    block_sync();
  }
  if (warp == 1) {
    if constexpr (kPair) tc::tmem_dealloc_pair(tmem, C::TMEM);
    else tc::tmem_dealloc(tmem, C::TMEM);
  }
}

constexpr int kNoShift = -(1 << 20);   // below any j

// --------------------------------------------------------------------------- small matrices

#include "ortho_small.cuh"

// ------------------------------------------------------------------------------------ host

// [rows x cols] fp16 in rows of `pitch` (a multiple of 64): boxes of 64 columns x 128 rows, or
// (chunked) of 2 x 64 columns x 64 rows, the columns in chunks of 64.
bool make_map(CUtensorMap* m, const __half* base, int rows, int cols, int pitch, bool chunked) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t ones[3] = {1u, 1u, 1u};
  CUresult r;
  if (chunked) {
    const cuuint64_t dims[3] = {64u, (cuuint64_t)rows, (cuuint64_t)(pitch / 64)};
    const cuuint64_t strides[2] = {(cuuint64_t)pitch * 2, 128u};
    const cuuint32_t box[3] = {64u, 64u, 2u};
    r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(base), dims, strides, box, ones,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  } else {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)pitch * 2};
    const cuuint32_t box[2] = {64u, 128u};
    r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<__half*>(base), dims, strides, box, ones,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  return r == CUDA_SUCCESS;
}

// A call's polynomial: coefficients, bounds, and how many steps the long matrices take on their
// small side before X is formed.
struct Plan {
  int steps = 0;
  double a[kMaxSteps], b[kMaxSteps], c[kMaxSteps];
  double u[kMaxSteps + 1], v[kMaxSteps];   // of the singular values before step k, of |M|
  // Where those of X_0 are at most 2^-j, step k's are at most 2^-j v_0 v_1 ... v_(k-1) too: X may be kept
  // times 2^max(0, j + shift_k), below the bound u_k that it is scaled to
  int shift[kMaxSteps + 1];
  std::vector<int> groups;
};
// The power of two that brings a matrix of this bound below 2^15.
double scale_of(double bound) { return std::exp2(std::floor(std::log2(32000.0 / bound))); }
constexpr double kMaxGrowth = 150.0;   // of L's rounding within a group
kfac_status make_plan(const kfac_ortho_desc* d, Plan* p) {
  p->steps = d->steps;
  double all_v = 1.0;
  double u = 1.0;   // bound of the singular values, a little above what exact arithmetic gives
  for (int k = 0; k < d->steps; ++k) {
    const double a = d->coefficients ? d->coefficients[3 * k] : 3.4445;
    const double b = d->coefficients ? d->coefficients[3 * k + 1] : -4.7750;
    const double c = d->coefficients ? d->coefficients[3 * k + 2] : 2.0315;
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return KFAC_ERR_INVALID_ARG;
    auto poly = [&](double t) { return std::fabs(a + b * t + c * t * t); };   // of t = sigma^2
    double v = std::max(poly(0.0), poly(u * u));
    if (c != 0.0) {
      const double t = -b / (2.0 * c);
      if (t > 0.0 && t < u * u) v = std::max(v, poly(t));
    }
    double next = u * poly(u * u);
    // where a + 3 b t + 5 c t^2 = 0
    const double disc = 9.0 * b * b - 20.0 * a * c;
    double at[2];
    int n = 0;
    if (c != 0.0 && disc >= 0.0) {
      at[n++] = (-3.0 * b + std::sqrt(disc)) / (10.0 * c);
      at[n++] = (-3.0 * b - std::sqrt(disc)) / (10.0 * c);
    } else if (c == 0.0 && b != 0.0) {
      at[n++] = -a / (3.0 * b);
    }
    for (int i = 0; i < n; ++i)
      if (at[i] > 0.0 && at[i] < u * u) next = std::max(next, std::sqrt(at[i]) * poly(at[i]));
    next *= 1.02;
    if (!(v >= 0x1p-20 && v <= 0x1p20 && next >= 0x1p-20 && next <= 0x1p20)) return KFAC_ERR_INVALID_ARG;
    p->a[k] = a;
    p->b[k] = b;
    p->c[k] = c;
    p->u[k] = u;
    p->v[k] = v;
    p->shift[k] = std::min(0, (int)std::floor(std::log2(u / all_v)));
    all_v *= v;
    u = next;
  }
  p->u[d->steps] = u;
  p->shift[d->steps] = kNoShift;   // the result is what it is
  for (int k = 0; k < d->steps;) {
    int g = 1;
    double growth = p->v[k] * p->v[k];
    while (k + g < d->steps && growth <= kMaxGrowth) {
      growth *= p->v[k + g] * p->v[k + g];
      ++g;
    }
    p->groups.push_back(g);
    k += g;
  }
  return KFAC_OK;
}

// Steps are grouped where X is long enough for that to pay: by operations from l > s on, measured later,
// since two launches more and products with fewer tiles come with it.  Single steps and groups, us, one
// matrix and eight, bf16: 1024 x 1536 158 and 186, 406 and 448; 1024 x 2048 170 and 191, 462 and 467;
// 2048 x 2560 301 and 313, 1274 and 1303; 2048 x 4096 336 and 329, 1744 and 1572; 4096 x 5120 1142 and
// 1134; 4096 x 8192 1564 and 1348.  Full arithmetic: 1024 x 2048 322 and 357, 2048 x 4096 792 and 718,
// 4096 x 8192 4816 and 3944.  So the border would better be near l = s + 1500 (512 x 4096 too: 189 and
// 174); up to there a matrix that this rule groups takes up to 18% longer.
bool grouped(int s, int l) { return s >= 1024 && l >= s + s / 2; }

enum { X_0, X_1, GRAM, TEMP, POLY, PROD_0, PROD_1, BUFFERS };
struct Matrix {
  int rows, cols, s, l, tall, group, xp, sp;    // pitches of X and of the s x s matrices
  int cluster;                                  // not 0: blocks of the small matrices' kernel
  size_t at[BUFFERS][2], part, r;               // [buffer][hi, lo]
};
// X_1 where X is formed more than once; two s x s matrices, five where steps are grouped
bool has_buffer(const Matrix& m, int steps, int b) {
  switch (b) {
    case X_0: case GRAM: case PROD_0: return true;
    case X_1: return steps > 1;
    default: return m.group;
  }
}
int64_t pitch_of(int64_t cols) { return cdiv(cols, 64) * 64; }

// One product of a matrix: buffers, scales; out BUFFERS: the call's result.
struct Op {
  int a, b, out, add;           // add: buffer or -1
  double alpha, beta, diag;
  int rpow, upper;
  int xpow, shift_in, shift_out;   // see Task
};
// A matrix's products, those of one entry at the same time.
std::vector<std::vector<Op>> ops_of(const Plan& p, bool group) {
  std::vector<std::vector<Op>> ops;
  std::vector<int> sizes = group ? p.groups : std::vector<int>(p.steps, 1);
  int x = X_0, k = 0;
  for (int g : sizes) {
    const bool first = k == 0, last = k + g == p.steps;
    const double sx = first ? 1.0 : scale_of(p.u[k]);   // X_0's factor is r, on the device
    double sl = scale_of(p.u[k] * p.u[k]);
    const int shift_in = p.shift[k];
    ops.push_back({{x, x, GRAM, -1, sl / (sx * sx), 0.0, 0.0, first ? 2 : 0, 1, 2, shift_in, kNoShift}});
    int prod = PROD_0;
    double sp = 1.0, bound = 1.0;
    for (int j = 0; j < g; ++j, ++k) {
      const double sm = scale_of(p.v[k]);
      const int poly = j == 0 ? PROD_0 : POLY;
      ops.push_back({{GRAM, GRAM, poly, GRAM, sm * p.c[k] / (sl * sl), sm * p.b[k] / sl, sm * p.a[k], 0, 1, 0, 0, 0}});
      std::vector<Op> both;
      bound *= p.v[k];
      if (j == 0) {
        sp = sm;
      } else {   // P <- M P
        const double to = scale_of(bound);
        const int next = prod == PROD_0 ? PROD_1 : PROD_0;
        both.push_back({POLY, prod, next, -1, to / (sm * sp), 0.0, 0.0, 0, 1, 0, 0, 0});
        prod = next;
        sp = to;
      }
      if (j + 1 < g) {   // L <- (L M) M
        const double st = scale_of(p.u[k] * p.u[k] * p.v[k]), to = scale_of(p.u[k + 1] * p.u[k + 1]);
        both.push_back({GRAM, poly, TEMP, -1, st / (sl * sm), 0.0, 0.0, 0, 1, 0, 0, 0});
        ops.push_back(both);
        ops.push_back({{TEMP, poly, GRAM, -1, to / (st * sm), 0.0, 0.0, 0, 1, 0, 0, 0}});
        sl = to;
      } else if (!both.empty()) {
        ops.push_back(both);
      }
    }
    const double to = last ? 1.0 : scale_of(p.u[k]);
    const int next = last ? BUFFERS : x == X_0 ? X_1 : X_0;
    ops.push_back({{prod, x, next, -1, to / (sp * sx), 0.0, 0.0, first ? 1 : 0, 0, 1, shift_in, p.shift[k]}});
    x = next;
  }
  return ops;
}

kfac_status check_sizes(const kfac_ortho_desc* d, int count, const int* rows, const int* cols) {
  if (!d || (d->dtype != KFAC_F32 && d->dtype != KFAC_BF16) ||
      (d->math != KFAC_ORTHO_FULL && d->math != KFAC_ORTHO_HALF))
    return KFAC_ERR_INVALID_ARG;
  if (d->steps < 1 || d->steps > kMaxSteps || !(d->eps >= 0.0) || !std::isfinite(d->eps) || count < 0)
    return KFAC_ERR_INVALID_ARG;
  if (count > 0 && (!rows || !cols)) return KFAC_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i)
    if (rows[i] < 0 || cols[i] < 0) return KFAC_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i)
    if (rows[i] > kMaxSide || cols[i] > kMaxSide) return KFAC_ERR_UNSUPPORTED;
  return KFAC_OK;
}

// Matrices that a product launch takes: up to two tasks each.  One more is a chain of launches by itself
// (512 x 512 in bf16: 24 take 223 us, 25 take 333; full arithmetic: 12 take 256, 13 take 446).
int per_launch(int halves) { return (halves == 2 ? Launch<true>::TASKS : Launch<false>::TASKS) / 2; }

// Blocks of the small matrices' kernel for a matrix; 0: too large for it.
int cluster_of(int s, int l, int halves) {
  return s > kSide ? 0 : halves == 2 ? small_cluster<true>(l) : small_cluster<false>(l);
}
// A matrix's regions of the workspace, from `at` on; returns where they end.
size_t lay_out_matrix(Matrix* m, int steps, int halves, size_t at) {
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes);
    return here;
  };
  m->xp = (int)pitch_of(m->cols);
  m->sp = (int)pitch_of(m->s);
  for (int b = 0; b < BUFFERS; ++b)
    for (int h = 0; h < halves && has_buffer(*m, steps, b); ++h)
      m->at[b][h] = take(b == X_0 || b == X_1 ? (size_t)m->rows * m->xp * 2 : (size_t)m->s * m->sp * 2);
  m->part = take(kPrepBlocks * 3 * sizeof(float));
  m->r = take(3 * sizeof(float));
  return at;
}
Matrix matrix_of(int rows, int cols, int steps) {
  Matrix m{};
  m.rows = rows;
  m.cols = cols;
  m.s = std::min(rows, cols);
  m.l = std::max(rows, cols);
  m.tall = rows > cols;
  m.group = steps > 1 && grouped(m.s, m.l);
  return m;
}
// What any of the matrices need, together or not: all the large ones, and as many of the small ones,
// the longest regions, as ever ride with them (lay_out).
size_t workspace_bytes(const kfac_ortho_desc* d, int count, const int* rows, const int* cols) {
  const int halves = d->math == KFAC_ORTHO_FULL ? 2 : 1, most = per_launch(halves) - 1;
  size_t bytes = 0, riding[kMaxGroup] = {};   // in falling order
  bool large = false;
  for (int i = 0; i < count; ++i) {
    Matrix m = matrix_of(rows[i], cols[i], d->steps);
    if (m.s == 0) continue;
    size_t n = lay_out_matrix(&m, d->steps, halves, 0);
    if (!cluster_of(m.s, m.l, halves)) {
      bytes += n;
      large = true;
      continue;
    }
    for (int k = 0; k < most; ++k)
      if (n > riding[k]) std::swap(n, riding[k]);
  }
  for (int k = 0; k < most && large; ++k) bytes += riding[k];
  return bytes;
}

// Regions of the workspace; matrices without elements take none and are left out.
size_t lay_out(const kfac_ortho_desc* d, int count, const int* rows, const int* cols,
               std::vector<Matrix>* out) {
  size_t at = 0;
  const int halves = d->math == KFAC_ORTHO_FULL ? 2 : 1;
  // Small matrices have a kernel of their own, unless the others' launches have room for them: there
  // they cost less, in the worst case the same.  Beside a large one, their own kernel and riding, us, bf16:
  // one 10 x 1024 beside 1024 x 1024 199 and 145; ten of 128 x 512 beside 300 x 300 148 and 109, beside
  // 4096 x 4096 997 and 987; ten of 128 x 4096 beside 1024 x 1024 236 and 235, beside 4096 x 4096 1042 and
  // 988; 23 of 64 x 64 beside 300 x 300 121 and 102.  Full arithmetic: one 10 x 1024 361 and 269, ten of
  // 128 x 1536 beside 1024 x 1024 387 and 336, eleven of 64 x 64 beside 300 x 300 197 and 164.
  int64_t small = 0, large = 0;
  for (int i = 0; i < count; ++i) {
    const int s = std::min(rows[i], cols[i]);
    if (s > 0) ++(cluster_of(s, std::max(rows[i], cols[i]), halves) ? small : large);
  }
  const int64_t room = cdiv(large, per_launch(halves)) * per_launch(halves) - large;
  for (int i = 0; i < count; ++i) {
    Matrix m = matrix_of(rows[i], cols[i], d->steps);
    if (m.s > 0 && small > room) m.cluster = cluster_of(m.s, m.l, halves);
    if (m.s > 0 && !m.cluster) at = lay_out_matrix(&m, d->steps, halves, at);
    out->push_back(m);
  }
  return at;
}

template <typename K> kfac_status allow_smem(OncePerDevice& once, K kern, size_t bytes) {
  int dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && once(dev, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) ==
               cudaSuccess;
      }))
    return KFAC_OK;
  check_launch();   // keeps the runtime's message
  return KFAC_ERR_CUDA;
}

template <int TO, typename T, bool kFull, bool kPair>
kfac_status launch_tiles(const Launch<kFull>& g, cudaStream_t st) {
  using C = Cfg<kFull, kPair>;
  static OncePerDevice once;
  if (kfac_status e = allow_smem(once, ortho_product_kernel<TO, T, kFull, kPair>, C::SMEM)) return e;
  if constexpr (kFull && kPair) {   // a register split that the launch does not cover would wait for ever
    cudaFuncAttributes at{};
    static OncePerDevice covered;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || !covered(dev, [&] {
          return cudaFuncGetAttributes(&at, ortho_product_kernel<TO, T, kFull, kPair>) == cudaSuccess &&
                 at.numRegs / 8 * 8 * C::THREADS >= 256 * kEpilogueRegs + 128 * kOtherRegs;
        })) {
      check_launch();
      return KFAC_ERR_UNSUPPORTED;
    }
  }
  constexpr int CTAS = kPair ? 2 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(CTAS * std::max(1, std::min(g.tile_start[g.count], num_sms() / CTAS))));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CTAS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, ortho_product_kernel<TO, T, kFull, kPair>, g);
  count_launch();
  return check_launch();
}
// Numbers the tasks' tiles and launches them: pairs on 256 x 256 tiles, or, where these would be
// fewer than half a tile per pair, single CTAs on 128 x 128 ones.  All launches of one matrix on singles and
// on pairs, us, bf16: 1024 x 1024 (10 tiles of 256 in L, 16 in X) 143 and 195; 1536 (21, 36) 183 and 233;
// 2048 (36, 64) 265 and 282, and 242 by this rule, L on singles and X on pairs; 2304 (45, 81) 449 and 357;
// 2560 (55, 100) 486 and 384.  Full arithmetic: 1536 353 and 525, 2048 544 and 649 (508 by the rule), 2304
// 999 and 901, 2560 1092 and 989.
template <int TO, typename T, bool kFull> kfac_status launch_product(Launch<kFull>& g, cudaStream_t st) {
  auto number = [&](int tile) {
    int64_t tiles = 0;
    for (int i = 0; i < g.count; ++i) {
      Task& t = g.task[i];
      t.tiles_m = (int)cdiv(t.M, tile);
      g.tile_start[i] = (int)tiles;
      tiles += t.upper ? (int64_t)t.tiles_m * (t.tiles_m + 1) / 2 : t.tiles_m * cdiv(t.N, tile);
    }
    g.tile_start[g.count] = (int)tiles;
    return tiles;
  };
  if (number(256) > num_sms() / 4) return launch_tiles<TO, T, kFull, true>(g, st);
  number(128);
  return launch_tiles<TO, T, kFull, false>(g, st);
}

// What a call works on, matrix by matrix.
struct Call {
  const kfac_ortho_desc* d;
  const void* const* x;
  const int64_t* ldx;
  void* const* out;             // orthogonalize
  const int64_t* ldo;
  float* const* momentum;       // step
  const int64_t* ldm;
  const kfac_ortho_step* hp;    // null: orthogonalize
};

// What the passes over x (and the momentum) need to know of matrix i of the call.
PrepTask prep_task(const Call& c, const Matrix& m, int i) {
  PrepTask t{};
  t.x = c.x[i];
  t.ldx = c.ldx[i];
  t.m = c.hp ? c.momentum[i] : nullptr;
  t.ldm = c.hp ? c.ldm[i] : 0;
  t.rows = m.rows;
  t.cols = m.cols;
  const int n = c.d->dtype == KFAC_BF16 ? 8 : 4;
  t.vec = m.cols % n == 0 && (uintptr_t)t.x % 16 == 0 && (m.rows == 1 || t.ldx % n == 0) &&
          (!c.hp || ((uintptr_t)t.m % 16 == 0 && (m.rows == 1 || t.ldm % 4 == 0)));
  const int pieces = (int)cdiv(m.cols, t.vec ? n : 1);
  t.tx = 1;
  while (t.tx < pieces && t.tx < kPrepThreads) t.tx *= 2;
  return t;
}
float rate_of(const kfac_ortho_step& hp, int rows, int cols) {
  return (float)(hp.lr * hp.update_scale * std::sqrt(std::max(1.0, (double)rows / (double)cols)));
}
float keep_of(const Call& c) { return (float)(1.0 - c.hp->lr * c.hp->weight_decay); }

// The product launch (small matrices: the step) whose first wait the thread's next call takes for one
// that ran out (kfac_selftest_orthogonal).
thread_local int t_selftest = -1;

template <int TO, typename TI, typename T, bool kFull>
kfac_status launch_small(const SmallLaunch& g, int count, cudaStream_t st) {
  static OncePerDevice once;
  using C = SmallCfg<kFull>;
  if (kfac_status e = allow_smem(once, ortho_small_kernel<TO, TI, T, kFull>,
                                 std::max(C::smem(C::most_tiles(1), 1), C::smem(C::most_tiles(8), 8))))
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(count * g.cluster));
  cfg.blockDim = dim3(kSmallThreads);
  cfg.dynamicSmemBytes = C::smem(g.tiles, g.cluster);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)g.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, ortho_small_kernel<TO, TI, T, kFull>, g);
  count_launch();
  return check_launch();
}

// The matrices with a side of at most kSide: a launch for each size of cluster.
template <bool kFull>
kfac_status run_small(const Call& c, const Plan& plan, const std::vector<Matrix>& ms, int give_up,
                      cudaStream_t st) {
  std::unique_ptr<SmallLaunch> g;
  for (int cs = 1; cs <= 8; cs *= 2) {
    for (size_t at = 0; at < ms.size();) {
      int n = 0, longest = 0;
      for (; at < ms.size() && n < kSmallTasks; ++at) {
        const Matrix& m = ms[at];
        if (m.cluster != cs || m.s == 0) continue;
        if (!g) g.reset(new SmallLaunch());
        SmallTask& t = g->task[n++];
        t.in = prep_task(c, m, (int)at);
        t.out = c.out[at];
        t.ldo = c.ldo[at];
        t.rate = c.hp ? rate_of(*c.hp, m.rows, m.cols) : 0.f;
        longest = std::max(longest, m.l);
      }
      if (n == 0) continue;
      g->steps = plan.steps;
      g->give_up = give_up;
      for (int k = 0; k < plan.steps; ++k) {   // ops_of, steps one by one
        const double sx = k == 0 ? 1.0 : scale_of(plan.u[k]), to = k + 1 == plan.steps ? 1.0 : scale_of(plan.u[k + 1]);
        const double sl = scale_of(plan.u[k] * plan.u[k]), sm = scale_of(plan.v[k]);
        g->step[k] = {(float)(sl / (sx * sx)), (float)(sm * plan.c[k] / (sl * sl)),
                      (float)(sm * plan.b[k] / sl), (float)(sm * plan.a[k]), (float)(to / (sm * sx)),
                      plan.shift[k], plan.shift[k + 1]};
      }
      g->cluster = cs;
      // a matrix's columns are divided by its own length alone: the sums' order is the same in any company
      g->tiles = cs == 1 ? (int)cdiv(longest, 64) : SmallCfg<kFull>::most_tiles(cs);
      g->nesterov = c.hp ? c.hp->nesterov : 0;
      g->mu = c.hp ? (float)c.hp->momentum : 0.f;
      g->eps = c.d->eps;
      g->keep = c.hp ? keep_of(c) : 1.f;
      kfac_status e;
      const bool bf16 = c.d->dtype == KFAC_BF16;
      if (c.hp)
        e = bf16 ? launch_small<TO_WEIGHTS, __nv_bfloat16, float, kFull>(*g, n, st)
                 : launch_small<TO_WEIGHTS, float, float, kFull>(*g, n, st);
      else
        e = bf16 ? launch_small<TO_OUT, __nv_bfloat16, __nv_bfloat16, kFull>(*g, n, st)
                 : launch_small<TO_OUT, float, float, kFull>(*g, n, st);
      if (e) return e;
    }
  }
  return KFAC_OK;
}

// The matrices of `idx` (at most half of a launch's tasks, none empty), all launches.
template <bool kFull>
kfac_status run_group(const Call& c, const Plan& plan, const std::vector<Matrix>& ms,
                      const std::vector<int>& idx, int give_up, char* ws, cudaStream_t st) {
  const int n = (int)idx.size();
  constexpr int halves = kFull ? 2 : 1;
  auto half_at = [&](size_t off) { return reinterpret_cast<__half*>(ws + off); };
  const bool bf16 = c.d->dtype == KFAC_BF16;
  const size_t es = bf16 ? 2 : 4;
  {
    std::unique_ptr<PrepLaunch> g(new PrepLaunch());
    int blocks = 0;
    for (int i = 0; i < n; ++i) {
      const Matrix& m = ms[idx[i]];
      PrepTask& t = g->task[i];
      t = prep_task(c, m, idx[i]);
      t.hi = half_at(m.at[X_0][0]);
      t.lo = kFull ? half_at(m.at[X_0][1]) : nullptr;
      t.part = reinterpret_cast<float*>(ws + m.part);
      t.r = reinterpret_cast<float*>(ws + m.r);
      t.pitch = m.xp;
      const int pieces = (int)cdiv(m.cols, t.vec ? 16 / (int)es : 1);
      g->block_start[i] = blocks;
      // 4 to 16 pieces a thread, by the matrix alone: its norm is summed the same in every company
      const int64_t rounds = cdiv((int64_t)m.rows, kPrepThreads / t.tx) * cdiv(pieces, t.tx);
      const int64_t each = std::max<int64_t>(4, std::min<int64_t>(16, rounds / 256));
      blocks += (int)std::min<int64_t>(kPrepBlocks, cdiv(rounds, each));
    }
    g->block_start[n] = blocks;
    g->count = n;
    g->mu = c.hp ? (float)c.hp->momentum : 0.f;
    g->nesterov = c.hp ? c.hp->nesterov : 0;
    g->eps = c.d->eps;
    const dim3 grid((unsigned)blocks), block(kPrepThreads);
    if (c.hp) {
      if (bf16) launch_pdl(ortho_norm_kernel<__nv_bfloat16, true>, grid, block, 0, st, *g);
      else launch_pdl(ortho_norm_kernel<float, true>, grid, block, 0, st, *g);
      if (bf16) launch_pdl(ortho_scale_kernel<__nv_bfloat16, true, kFull>, grid, block, 0, st, *g);
      else launch_pdl(ortho_scale_kernel<float, true, kFull>, grid, block, 0, st, *g);
    } else {
      if (bf16) launch_pdl(ortho_norm_kernel<__nv_bfloat16, false>, grid, block, 0, st, *g);
      else launch_pdl(ortho_norm_kernel<float, false>, grid, block, 0, st, *g);
      if (bf16) launch_pdl(ortho_scale_kernel<__nv_bfloat16, false, kFull>, grid, block, 0, st, *g);
      else launch_pdl(ortho_scale_kernel<float, false, kFull>, grid, block, 0, st, *g);
    }
    count_launch(2);
    if (kfac_status e = check_launch()) return e;
  }
  // every buffer's maps, once, in both kinds of boxes
  struct Maps {
    CUtensorMap of[BUFFERS][2][2];   // [hi, lo][rows, chunks]
  };
  std::vector<Maps> maps(n);
  std::vector<std::vector<std::vector<Op>>> ops(n);
  size_t rounds = 0;
  for (int i = 0; i < n; ++i) {
    const Matrix& m = ms[idx[i]];
    for (int b = 0; b < BUFFERS; ++b) {
      const bool x = b == X_0 || b == X_1;
      for (int h = 0; h < halves && has_buffer(m, plan.steps, b); ++h)
        for (int k = 0; k < (x ? 2 : 1); ++k)   // (only an X is read as MN-major tiles)
          if (!make_map(&maps[i].of[b][h][k], half_at(m.at[b][h]), x ? m.rows : m.s, x ? m.cols : m.s,
                        x ? m.xp : m.sp, k))
            return KFAC_ERR_CUDA;
    }
    ops[i] = ops_of(plan, m.group);
    rounds = std::max(rounds, ops[i].size());
  }
  // the matrices' products side by side, the last ones of all together in the last launch
  std::unique_ptr<Launch<kFull>> g(new Launch<kFull>());
  for (size_t round = 0; round < rounds; ++round) {
    g->count = 0;
    g->give_up = (int)round == give_up;
    const bool last = round + 1 == rounds;
    for (int i = 0; i < n; ++i) {
      if (round + ops[i].size() < rounds) continue;
      const Matrix& m = ms[idx[i]];
      for (const Op& op : ops[i][round + ops[i].size() - rounds]) {
        Task& t = g->task[g->count];
        CUtensorMap* to = g->maps[g->count++];
        t = Task{};
        t.r = reinterpret_cast<float*>(ws + m.r);
        t.alpha = (float)op.alpha;
        t.beta = (float)op.beta;
        t.diag = (float)op.diag;
        t.rpow = op.rpow;
        t.xpow = op.xpow;
        t.shift_in = op.shift_in;
        t.shift_out = op.shift_out;
        t.upper = op.upper;
        t.same_ab = op.a == op.b;
        int a = op.a, b = op.b;
        if (op.upper) {
          const bool x = a == X_0 || a == X_1;   // L = X X^T, or X^T X of a tall X
          t.M = t.N = m.s;
          t.kblocks = (int)cdiv(x ? m.l : m.s, 64);
          t.mn_a = t.mn_b = x && m.tall;
        } else {                                 // P X, or X P of a tall X (P is symmetric)
          t.M = m.rows;
          t.N = m.cols;
          t.kblocks = (int)cdiv(m.s, 64);
          if (m.tall) std::swap(a, b);
          else t.mn_b = 1;
        }
        if (op.add >= 0) {
          t.add_hi = half_at(m.at[op.add][0]);
          t.add_lo = kFull ? half_at(m.at[op.add][1]) : nullptr;
          t.add_pitch = m.sp;
        }
        for (int h = 0; h < halves; ++h) {
          to[h * MAPS + MAP_A] = maps[i].of[a][h][t.mn_a];
          to[h * MAPS + MAP_B] = maps[i].of[b][h][t.mn_b];
          if (op.out < BUFFERS) {
            to[h * MAPS + MAP_STORE] = maps[i].of[op.out][h][0];
          }
        }
        if (op.upper) {
          t.mirror_hi = half_at(m.at[op.out][0]);
          t.mirror_lo = kFull ? half_at(m.at[op.out][1]) : nullptr;
          t.mirror_pitch = m.sp;
        }
        if (op.out == BUFFERS) {
          t.out = c.out[idx[i]];
          t.out_ld = c.ldo[idx[i]];
          if (c.hp) {
            t.keep = keep_of(c);
            t.rate = rate_of(*c.hp, m.rows, m.cols);
          }
        }
      }
    }
    kfac_status e;
    if (!last) e = launch_product<TO_MATRIX, float, kFull>(*g, st);
    else if (c.hp) e = launch_product<TO_WEIGHTS, float, kFull>(*g, st);
    else if (bf16) e = launch_product<TO_OUT, __nv_bfloat16, kFull>(*g, st);
    else e = launch_product<TO_OUT, float, kFull>(*g, st);
    if (e) return e;
  }
  return KFAC_OK;
}

kfac_status run(const Call& c, int count, const int* rows, const int* cols, void* workspace,
                size_t bytes, cudaStream_t st) {
  const int give_up = t_selftest;
  t_selftest = -1;
  Plan plan;
  if (kfac_status e = make_plan(c.d, &plan)) return e;
  std::vector<Matrix> ms;
  const size_t need = lay_out(c.d, count, rows, cols, &ms);
  if (need && (!workspace || (uintptr_t)workspace % kAlign || bytes < need)) return KFAC_ERR_WORKSPACE;
  // longest reductions first: the last round of tiles then holds the shortest
  std::vector<int> order;
  for (int i = 0; i < count; ++i)
    if (ms[i].s > 0 && !ms[i].cluster) order.push_back(i);
  if (kfac_status e = c.d->math == KFAC_ORTHO_FULL ? run_small<true>(c, plan, ms, give_up, st)
                                                   : run_small<false>(c, plan, ms, give_up, st))
    return e;
  std::stable_sort(order.begin(), order.end(), [&](int a, int b) { return ms[a].l > ms[b].l; });
  const bool full = c.d->math == KFAC_ORTHO_FULL;
  const size_t most = (size_t)per_launch(full ? 2 : 1);
  for (size_t at = 0; at < order.size(); at += most) {
    const std::vector<int> idx(order.begin() + at, order.begin() + std::min(order.size(), at + most));
    kfac_status e = full
                        ? run_group<true>(c, plan, ms, idx, give_up, static_cast<char*>(workspace), st)
                        : run_group<false>(c, plan, ms, idx, give_up, static_cast<char*>(workspace), st);
    if (e) return e;
  }
  return KFAC_OK;
}

bool bad_matrix(const void* p, int64_t ld, int rows, int cols, size_t es) {
  return !p || (uintptr_t)p % es || ld < 0 || ld > (int64_t(1) << 40) || (rows > 1 && ld < cols);
}

// Addresses of the matrices with elements, sorted, with their indexes.
using Places = std::vector<std::pair<const void*, int>>;
template <typename Q> Places places(Q const* p, int count, const int* rows, const int* cols) {
  Places at;
  for (int i = 0; i < count; ++i)
    if (rows[i] > 0 && cols[i] > 0) at.emplace_back(p[i], i);
  std::sort(at.begin(), at.end());
  return at;
}
// Whether two matrices are the same one (their results would depend on which came last).
bool any_twice(const Places& p) {
  return std::adjacent_find(p.begin(), p.end(), [](auto& a, auto& b) { return a.first == b.first; }) != p.end();
}
// Whether a result (no two the same) lies where something else is read, other than as may(i) allows: the
// matrix's own.
template <typename F> bool any_shared(const Places& results, const Places& others, F may) {
  for (auto& o : others) {
    auto r = std::lower_bound(results.begin(), results.end(), std::make_pair(o.first, -1));
    if (r != results.end() && r->first == o.first && (r->second != o.second || !may(o.second))) return true;
  }
  return false;
}

// A C entry lets no exception out: what can be thrown here is a failed host allocation.
template <typename F> kfac_status guarded(F f) {
  try {
    return f();
  } catch (...) {
    return KFAC_ERR_CUDA;
  }
}

}  // namespace

// The first device-side error of these kernels since the last call, cleared.
kfac_status take_status(DevStatus* s) {
  const DevStatus zero{};
  if (cudaMemcpyFromSymbol(s, g_status, sizeof(*s)) != cudaSuccess) return KFAC_ERR_CUDA;
  if (s->code && cudaMemcpyToSymbol(g_status, &zero, sizeof(zero)) != cudaSuccess) return KFAC_ERR_CUDA;
  return KFAC_OK;
}

}  // namespace ortho
}  // namespace kfac

using namespace kfac;
using namespace kfac::ortho;

extern "C" kfac_status kfac_orthogonalize_workspace_size(const kfac_ortho_desc* d, int count,
                                                         const int* rows, const int* cols,
                                                         size_t* bytes) {
  if (!bytes) return KFAC_ERR_INVALID_ARG;
  if (kfac_status e = check_sizes(d, count, rows, cols)) return e;
  *bytes = workspace_bytes(d, count, rows, cols);
  return KFAC_OK;
}

extern "C" kfac_status kfac_orthogonalize(const kfac_ortho_desc* d, int count, const int* rows,
                                          const int* cols, const void* const* x, const int64_t* ldx,
                                          void* const* out, const int64_t* ldo, void* workspace,
                                          size_t workspace_bytes, cudaStream_t stream) {
  if (kfac_status e = check_sizes(d, count, rows, cols)) return e;
  if (count == 0) return KFAC_OK;
  if (!x || !ldx || !out || !ldo) return KFAC_ERR_INVALID_ARG;
  const size_t es = d->dtype == KFAC_BF16 ? 2 : 4;
  for (int i = 0; i < count; ++i) {
    if (rows[i] == 0 || cols[i] == 0) continue;
    if (bad_matrix(x[i], ldx[i], rows[i], cols[i], es) || bad_matrix(out[i], ldo[i], rows[i], cols[i], es))
      return KFAC_ERR_INVALID_ARG;
  }
  Call c{};
  c.d = d;
  c.x = x;
  c.ldx = ldx;
  c.out = out;
  c.ldo = ldo;
  return guarded([&] {
    const Places results = places(out, count, rows, cols);
    if (any_twice(results) || any_shared(results, places(x, count, rows, cols),
                                         [&](int i) { return rows[i] == 1 || ldx[i] == ldo[i]; }))
      return KFAC_ERR_INVALID_ARG;
    return run(c, count, rows, cols, workspace, workspace_bytes, stream);
  });
}

extern "C" kfac_status kfac_orthogonal_step(const kfac_ortho_desc* d, const kfac_ortho_step* hp, int count,
                                            const int* rows, const int* cols, const void* const* grad,
                                            const int64_t* ldg, float* const* momentum,
                                            const int64_t* ldm, float* const* param, const int64_t* ldp,
                                            void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (kfac_status e = check_sizes(d, count, rows, cols)) return e;
  if (!hp || !std::isfinite(hp->lr) || !std::isfinite(hp->momentum) || !std::isfinite(hp->weight_decay) ||
      !std::isfinite(hp->update_scale) || (hp->nesterov != 0 && hp->nesterov != 1))
    return KFAC_ERR_INVALID_ARG;
  if (count == 0) return KFAC_OK;
  if (!grad || !ldg || !momentum || !ldm || !param || !ldp) return KFAC_ERR_INVALID_ARG;
  const size_t es = d->dtype == KFAC_BF16 ? 2 : 4;
  if (!std::isfinite((float)hp->momentum) || !std::isfinite((float)(1.0 - hp->lr * hp->weight_decay)))
    return KFAC_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    if (rows[i] == 0 || cols[i] == 0) continue;
    if (!std::isfinite(rate_of(*hp, rows[i], cols[i]))) return KFAC_ERR_INVALID_ARG;
    if (bad_matrix(grad[i], ldg[i], rows[i], cols[i], es) ||
        bad_matrix(momentum[i], ldm[i], rows[i], cols[i], 4) ||
        bad_matrix(param[i], ldp[i], rows[i], cols[i], 4))
      return KFAC_ERR_INVALID_ARG;
  }
  return guarded([&] {
    std::vector<void*> out(param, param + count);
    const Places g = places(grad, count, rows, cols), m = places(momentum, count, rows, cols),
                 w = places(param, count, rows, cols);
    auto never = [](int) { return false; };
    if (any_twice(w) || any_twice(m) || any_shared(w, m, never) || any_shared(w, g, never) ||
        any_shared(m, g, never))
      return KFAC_ERR_INVALID_ARG;
    Call c{};
    c.d = d;
    c.x = grad;
    c.ldx = ldg;
    c.out = out.data();
    c.ldo = ldp;
    c.momentum = momentum;
    c.ldm = ldm;
    c.hp = hp;
    return run(c, count, rows, cols, workspace, workspace_bytes, stream);
  });
}

extern "C" kfac_status kfac_selftest_orthogonal(int launch) {
  if (launch < -1) return KFAC_ERR_INVALID_ARG;
  t_selftest = launch;
  return KFAC_OK;
}
