// Orthogonalised updates by Newton-Schulz products.  Of a matrix G with small side s and long
// side l (X stands for G or, by its columns, for G^T):
//   X_0 = G / (|G|_F + eps);   L = X X^T,  M = a I + b L + c L^2,  X <- M X   per step,
// after which the singular values of X are near one (a polynomial of each: a t + b t^3 + c t^5).
//
// Per step two symmetric products (s^2 l and s^3 multiply-adds over their distinct halves) and one
// whole one (s^2 l): bound by the tensor cores where there are tiles for every SM, by the chain of
// 3 steps launches where there are not.
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
// One kernel serves the three products: CTA pairs (tcgen05 cta_group::2) on 256 x 256 tiles of all
// the call's matrices, persistent, a warp for TMA, one for the MMAs, eight for the epilogue, two
// accumulators in TMEM so that a tile's epilogue runs beside the next one's products.  A matrix
// is never transposed: the operand whose k runs down the rows of X is read as it lies, as an
// MN-major tile.  Of a symmetric product the tiles on and above the diagonal are computed; the
// epilogue stores each of them and its transpose through shared memory by TMA.
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
#include <numeric>
#include <vector>

namespace kfac {
namespace ortho {

__device__ DevStatus g_status;   // device-side errors, read by kfac_operator_status

namespace {

constexpr int kMaxGroup = 32;        // matrices per launch
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
  float* r;
  int rows, cols, pitch;
  int tx;                  // threads per row (a power of two)
  int vec;                 // whole 16-byte vectors of x (and of m)
};
struct PrepLaunch {
  PrepTask task[kMaxGroup];
  int block_start[kMaxGroup + 1];
  int count;
  float mu, eps;
  int nesterov;
};

__device__ __forceinline__ int task_of(const int* start, int count, int block) {
  int q = 0;
  while (q + 1 < count && block >= start[q + 1]) ++q;
  return q;
}

template <typename T, int N> struct alignas(N * sizeof(T)) Vec { T v[N]; };

// Squares in three ranges, so that none of 2^30 overflows or vanishes: of values from 2^40 (scaled
// by 2^-84), below 2^-40 (by 2^88: from 2^-149 on), and the others.
struct Squares {
  float big = 0.f, mid = 0.f, small = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float m = fabsf(v);
    if (m < 0x1p-40f) {
      const float t = v * 0x1p88f;
      small = fmaf(t, t, small);
    } else if (m < 0x1p40f) {
      mid = fmaf(v, v, mid);
    } else {   // Inf and NaN too
      const float t = v * 0x1p-84f;
      big = fmaf(t, t, big);
    }
  }
};

// N values of the matrix to orthogonalise from column c of a row: x, or with the momentum
// m <- mu m + g the update g + mu m (nesterov) or m.  kStore: m is written.
template <typename T, int N, bool kStep, bool kStore>
__device__ __forceinline__ void load_update(const PrepLaunch& g, const PrepTask& t, int64_t row, int c,
                                            float (&u)[N]) {
  const Vec<T, N> p = *reinterpret_cast<const Vec<T, N>*>(static_cast<const T*>(t.x) + row * t.ldx + c);
#pragma unroll
  for (int i = 0; i < N; ++i) u[i] = to_f32<T>(p.v[i]);
  if constexpr (kStep) {
    constexpr int F = N < 4 ? N : 4;
    float* m = t.m + row * t.ldm + c;
#pragma unroll
    for (int j = 0; j < N; j += F) {
      Vec<float, F> v = *reinterpret_cast<const Vec<float, F>*>(m + j);
      if (kStore) {
#pragma unroll
        for (int i = 0; i < F; ++i) v.v[i] = fmaf(g.mu, v.v[i], u[j + i]);
        *reinterpret_cast<Vec<float, F>*>(m + j) = v;
      }
#pragma unroll
      for (int i = 0; i < F; ++i) u[j + i] = g.nesterov ? fmaf(g.mu, v.v[i], u[j + i]) : v.v[i];
    }
  }
}

template <typename F> __device__ __forceinline__ void each_row_piece(const PrepTask& t, int n, int block,
                                                                    int blocks, F f) {
  const int tc = threadIdx.x % t.tx, tr = threadIdx.x / t.tx, rpb = kPrepThreads / t.tx;
  for (int64_t row = (int64_t)block * rpb + tr; row < t.rows; row += (int64_t)blocks * rpb)
    for (int c = tc * n; c < t.cols; c += t.tx * n) f(row, c);
}

template <typename T, bool kStep>
__global__ void __launch_bounds__(kPrepThreads) ortho_norm_kernel(const __grid_constant__ PrepLaunch g) {
  __shared__ float red[3][kPrepThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int q = task_of(g.block_start, g.count, blockIdx.x);
  const PrepTask& t = g.task[q];
  const int block = blockIdx.x - g.block_start[q], blocks = g.block_start[q + 1] - g.block_start[q];
  constexpr int N = 16 / (int)sizeof(T);
  Squares s;
  if (t.vec) {
    each_row_piece(t, N, block, blocks, [&](int64_t row, int c) {
      float u[N];
      load_update<T, N, kStep, true>(g, t, row, c, u);
#pragma unroll
      for (int i = 0; i < N; ++i) s.add(u[i]);
    });
  } else {
    each_row_piece(t, 1, block, blocks, [&](int64_t row, int c) {
      float u[1];
      load_update<T, 1, kStep, true>(g, t, row, c, u);
      s.add(u[0]);
    });
  }
  float v[3] = {s.big, s.mid, s.small};
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

// X_0 = x 2^k with |X_0|_F in (2^13, 2^14], and r with x / (|x| + eps) = r X_0.
template <typename T, bool kStep, bool kFull>
__global__ void __launch_bounds__(kPrepThreads) ortho_scale_kernel(const __grid_constant__ PrepLaunch g) {
  __shared__ double sums[3];
  __shared__ float factor[2];   // 2^k in two, each within fp32's range
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
    const double norm = sqrt(sums[0] * 0x1p168 + sums[1] + sums[2] * 0x1p-176) + (double)g.eps;
    float r = 0.f;
    int k = 0;
    if (norm > 0.0 && isfinite(norm)) {
      int e = 0;
      frexp(norm, &e);                         // norm < 2^e
      k = 14 - e;
      r = (float)ldexp(1.0 / norm, -k);
    } else if (norm != 0.0) {                  // Inf and NaN reach everything through r
      r = __int_as_float(0x7fffffff);
    }
    const int k0 = min(max(k, -126), 126);
    factor[0] = ldexpf(1.f, k0);
    factor[1] = ldexpf(1.f, k - k0);
    if (block == 0) *t.r = r;
  }
  __syncthreads();
  const float up0 = factor[0], up1 = factor[1];
  constexpr int N = 16 / (int)sizeof(T);
  auto store = [&](auto& u, int64_t row, int c) {
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
  if (t.vec) {
    each_row_piece(t, N, block, blocks, [&](int64_t row, int c) {
      float u[N];
      load_update<T, N, kStep, false>(g, t, row, c, u);
      store(u, row, c);
    });
  } else {
    each_row_piece(t, 1, block, blocks, [&](int64_t row, int c) {
      float u[1];
      load_update<T, 1, kStep, false>(g, t, row, c, u);
      store(u, row, c);
    });
  }
}

// -------------------------------------------------------------------------------- products

enum { PH_GRAM, PH_POLY, PH_APPLY, PH_OUT, PH_STEP };   // L, M, X, the last X, and with it W

// out = alpha r^rpow A B^T [+ beta add + diag I], stored as fp16 (or PH_OUT, PH_STEP below)
struct Task {
  int64_t out_ld;
  void* out;                    // PH_OUT: the direction; PH_STEP: the weights, fp32
  const __half *add_hi, *add_lo;   // PH_POLY: L
  const float* r;
  float alpha, beta, diag;
  float keep, rate;             // PH_STEP: W <- keep W - rate X
  int rpow, add_pitch;
  int M, N, kblocks;            // sizes of the product; k in blocks of 64
  int tiles_m, tiles_n, upper;  // upper: symmetric, tiles on and above the diagonal
  int mn_a, mn_b;               // operands read as MN-major tiles
};
template <bool kFull> struct Launch {
  // operand A, operand B, direct store; mirror store in B's place where A is B (GRAM, POLY)
  CUtensorMap maps[kMaxGroup][kFull ? 6 : 3];
  Task task[kMaxGroup];
  int tile_start[kMaxGroup + 1];
  int count;
};

template <bool kFull> struct Cfg {
  static constexpr int BK = 64;
  static constexpr int HALF = 128 * BK * 2;              // 128 rows (or features) of an operand
  static constexpr int STAGE = HALF * 2 * (kFull ? 2 : 1);
  static constexpr int STAGES = kFull ? 3 : 5;
  static constexpr int NBUF = kFull ? 1 : 2;             // 16 KB store buffers per epilogue group
  static constexpr int BUF = 128 * 64 * 2;
  static constexpr int SUB = kFull ? 1 : 1 << 20;        // k blocks per drain
  static constexpr int EPI_WARPS = 8, THREADS = 64 + 32 * EPI_WARPS;
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE + 2 * NBUF * BUF + 512;
  static_assert(SMEM <= 232448, "fits the per-CTA shared memory");
};

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
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(tc::smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(src))
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

// Tile t of the launch: its matrix, row and column block.
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
// Transposed: two blocks (rows 0-63, 64-127) of 64 columns x 64 rows.  Neighbouring lanes trade
// values so that each writes whole words, of columns c and c + 4, which fall on different banks.
__device__ __forceinline__ void put_columns(uint8_t* buf, int row, const uint32_t (&w)[32]) {
  const bool odd = row & 1;
  uint8_t* block = buf + (row >> 6) * 8192;
  const int e = row & 62;   // the even row of the pair, within the block
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // columns c = 2 (j + k) + {0, 1} and c + 4
      const uint32_t lo = w[j + k], hi = w[j + k + 2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int c = 2 * (j + k) + b;
        const uint32_t p = __byte_perm(lo, hi, b ? 0x7632 : 0x5410);   // (column c, column c + 4)
        const uint32_t o = __shfl_xor_sync(0xffffffffu, p, 1);
        const uint32_t word = odd ? __byte_perm(p, o, 0x3276) : __byte_perm(p, o, 0x5410);
        const int cc = odd ? c + 4 : c;
        *reinterpret_cast<uint32_t*>(block + cc * 128 + (((e >> 3) ^ (cc & 7)) << 4) + (e & 7) * 2) = word;
      }
    }
  }
}

template <int PH, typename TO, bool kFull>
__global__ void __launch_bounds__(Cfg<kFull>::THREADS, 1)
    ortho_product_kernel(const __grid_constant__ Launch<kFull> g) {
  using C = Cfg<kFull>;
  constexpr int STAGES = C::STAGES;
  constexpr bool kSym = PH == PH_GRAM || PH == PH_POLY, kLast = PH == PH_OUT || PH == PH_STEP;
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
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int total = g.tile_start[g.count];
  const uint32_t rank = tc::cluster_rank();
  const int pair = (int)(blockIdx.x / 2), npairs = (int)(gridDim.x / 2);
  // a role that gives up stops the peer CTA's roles too
  const uint32_t peer_abort = tc::mapa((const void*)abort_flag, rank ^ 1u);
  auto give_up = [&](int info) {
    report_error(&g_status, KFAC_ERR_TIMEOUT, -1, info);
    *abort_flag = 1;
    tc::st_cluster_u32(peer_abort, 1u);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&acc_full[b], 1);
      tc::mbar_init(&acc_empty[b], 2 * C::EPI_WARPS);
    }
    tc::mbar_init(drained, 1);
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc_pair(tmem_slot, 512);
    tc::tmem_relinquish_pair();
  }
  tc::tc_fence_before();
  __syncwarp();
  tc::cluster_sync();   // both CTAs' barriers initialised and TMEM allocated
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  // a diagonal tile of a symmetric product: this CTA's rows of A are its half of B
  auto shared_ab = [&](int ti, int tj) { return kSym && ti == tj; };

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      const uint32_t full0 = tc::mapa(full, 0);   // the even CTA's stage barriers
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = pair; t < total && ok; t += npairs) {
        int q, ti, tj;
        tile_of(g, t, &q, &ti, &tj);
        const Task& k = g.task[q];
        const bool ab = shared_ab(ti, tj);
        const int arow = ti * 256 + (int)rank * 128, brow = tj * 256 + (int)rank * 128;
        const CUtensorMap *ma = &g.maps[q][0], *mb = kSym ? ma : &g.maps[q][1];
        constexpr int LO = 3;   // the lo halves' maps
        for (int kb = 0; kb < k.kblocks; ++kb) {
          if (!tc::mbar_wait(&empty[stage], phase ^ 1, abort_flag)) {
            give_up(41);
            ok = false;
            break;
          }
          const uint32_t fb = full0 + (uint32_t)(stage * sizeof(uint64_t));
          if (rank == 0)
            tc::mbar_expect_tx(&full[stage], 2 * (ab ? C::STAGE / 2 : C::STAGE));   // both CTAs' loads
          uint8_t* at = smem + (size_t)stage * C::STAGE;
          auto load = [&](uint8_t* dst, const CUtensorMap* m, int mn, int row) {
            if (mn) tc::tma_load_3d_pair(dst, m, fb, 0, kb * C::BK, row / 64);
            else tc::tma_load_2d_pair(dst, m, fb, kb * C::BK, row);
          };
#pragma unroll
          for (int part = 0; part < (kFull ? 2 : 1); ++part) {
            if (!ab) load(at + part * 2 * C::HALF, ma + part * LO, k.mn_a, arow);
            load(at + part * 2 * C::HALF + C::HALF, mb + part * LO, k.mn_b, brow);
          }
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // A CTA that gave up lets its memory go only after its copies have landed: they complete on
      // the even CTA's barriers, which it waits for (bounded) before both leave.
      if (*abort_flag && rank == 0) {
        volatile int never = 0;
        for (int s = 0; s < STAGES; ++s)
          if (const int uses = ring_uses(issued, s, STAGES))
            tc::mbar_wait(&full[s], ring_last_parity(uses), &never);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (rank == 0) {
      const uint32_t leader = tc::elect_leader();
      int stage = 0, gsub = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = pair; t < total && ok; t += npairs) {
        int q, ti, tj;
        tile_of(g, t, &q, &ti, &tj);
        const bool ab = shared_ab(ti, tj);
        const int kblocks = g.task[q].kblocks, mn_a = g.task[q].mn_a, mn_b = g.task[q].mn_b;
        const uint32_t idesc = tc::make_idesc(0, 256, 256) | (mn_a ? tc::kIdescMnA : 0) |
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
          const uint32_t d = tmem + (uint32_t)(buf * 256);
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
                umma_pair_by(leader, d, ak, bk + LO, idesc, kb > kb0 || kk > 0);
                umma_pair_by(leader, d, ak + LO, bk, idesc, 1u);
              }
            }
#pragma unroll
            for (int kk = 0; kk < C::BK / 16; ++kk)
              umma_pair_by(leader, d, a + kk * step_a, b + kk * step_b, idesc, kFull || kb > kb0 || kk > 0);
            commit_pair_by(leader, &empty[stage]);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (ok) commit_pair_by(leader, &acc_full[buf]);
        }
      }
      if (!ok || *abort_flag) {   // the products in flight end before TMEM and the tiles go
        commit_pair_by(leader, drained);
        volatile int never = 0;
        tc::mbar_wait(drained, 0, &never);
      }
    }
  } else {
    // -------------------------------------------------------------------- epilogue
    const int qd = warp & 3;                 // TMEM lane quarter this warp may access
    const int h = (warp - 2) >> 2;           // columns [128 h, 128 h + 128) of the tile
    const int row = 32 * qd + lane;
    const bool issuer = warp == 2 + 4 * h && lane == 0;
    uint8_t* mybufs = bufs + h * C::NBUF * C::BUF;
    const uint32_t acc_empty0 = tc::mapa(acc_empty, 0);
    int gsub = 0, turn = 0;
    bool ok = true;
    for (int t = pair; t < total; t += npairs) {
      int q, ti, tj;
      tile_of(g, t, &q, &ti, &tj);
      const Task& k = g.task[q];
      const int r0 = ti * 256 + (int)rank * 128, gr = r0 + row;
      const int nsub = (k.kblocks + C::SUB - 1) / C::SUB;
      float alpha = k.alpha;
      if (k.rpow) {
        const float r = __ldg(k.r);
        alpha *= k.rpow == 2 ? r * r : r;
      }
      float sum[kFull ? 128 : 1];
      if constexpr (kFull) {
#pragma unroll
        for (int i = 0; i < 128; ++i) sum[i] = 0.f;
        for (int sub = 0; sub < nsub && ok; ++sub, ++gsub) {
          const int buf = gsub & 1, use = gsub >> 1;
          if (!tc::mbar_wait(&acc_full[buf], use & 1, abort_flag)) {
            if (lane == 0) give_up(44);
            ok = false;
            break;
          }
          tc::tc_fence_after();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float v[32];
            tc::tmem_ld32(tmem + ((uint32_t)(32 * qd) << 16) + (uint32_t)(buf * 256 + h * 128 + c * 32), v);
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[c * 32 + i] += v[i];
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive_remote(acc_empty0 + (uint32_t)(buf * sizeof(uint64_t)));
        }
      } else if (ok) {
        if (!tc::mbar_wait(&acc_full[gsub & 1], (gsub >> 1) & 1, abort_flag)) {
          if (lane == 0) give_up(45);
          ok = false;
        }
        tc::tc_fence_after();
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok && PH != PH_OUT) break;        // PH_OUT: the tiles from here on become NaN
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {       // 64 columns at a time
        const int c0 = tj * 256 + h * 128 + ch * 64;
        float v[64];
        if constexpr (kFull) {
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i] = sum[ch * 64 + i] * alpha;
        } else {
          if (ok) {
            uint32_t w0[32], w1[32];
            const uint32_t at =
                tmem + ((uint32_t)(32 * qd) << 16) + (uint32_t)((gsub & 1) * 256 + h * 128 + ch * 64);
            tc::tmem_ld32_issue(at, w0);
            tc::tmem_ld32_issue(at + 32, w1);
            tc::tmem_ld_wait();
            tc::tmem_ld_use(w0);
            tc::tmem_ld_use(w1);
            if (ch == 1) {
              tc::tc_fence_before();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive_remote(acc_empty0 + (uint32_t)((gsub & 1) * sizeof(uint64_t)));
            }
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
        if (c0 >= k.N || r0 >= k.M) continue;   // (the whole group)
        if constexpr (kLast) {
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
            const int rows = min(32, k.M - (r0 + 32 * qd));
            TO* out = static_cast<TO*>(k.out) + (int64_t)(r0 + 32 * qd) * k.out_ld + c;
            if (c < k.N) {
#pragma unroll 8
              for (int i = 0; i < rows; ++i) {
                float x = mine[i * 32 + (((lane >> 2) ^ (i & 7)) << 2) + (lane & 3)];
                if constexpr (PH == PH_STEP) {
                  const float w = to_f32<TO>(out[(int64_t)i * k.out_ld]);
                  x = fmaf(-k.rate, x, k.keep * w);
                } else if (!ok) {
                  x = __int_as_float(0x7fffffff);
                }
                out[(int64_t)i * k.out_ld] = (TO)x;
              }
            }
          }
        } else {
          if constexpr (PH == PH_POLY) {
            if (gr < k.M) {
              const __half* add = k.add_hi + (int64_t)gr * k.add_pitch + c0;
              const __half* add_lo = kFull ? k.add_lo + (int64_t)gr * k.add_pitch + c0 : nullptr;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const uint4 w = *reinterpret_cast<const uint4*>(add + 8 * j);
                const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 f = unpack2(e[i]);
                  v[8 * j + 2 * i] = fmaf(k.beta, f.x, v[8 * j + 2 * i]);
                  v[8 * j + 2 * i + 1] = fmaf(k.beta, f.y, v[8 * j + 2 * i + 1]);
                }
                if constexpr (kFull) {
                  const uint4 wl = *reinterpret_cast<const uint4*>(add_lo + 8 * j);
                  const uint32_t el[4] = {wl.x, wl.y, wl.z, wl.w};
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack2(el[i]);
                    v[8 * j + 2 * i] = fmaf(k.beta, f.x, v[8 * j + 2 * i]);
                    v[8 * j + 2 * i + 1] = fmaf(k.beta, f.y, v[8 * j + 2 * i + 1]);
                  }
                }
              }
            }
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (c0 + i == gr) v[i] += k.diag;
          }
          // hi (and lo) values, each as they are and, off the diagonal, transposed
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
#pragma unroll
            for (int mirror = 0; mirror < (kSym ? 2 : 1); ++mirror) {
              if (mirror && ti == tj) continue;
              uint8_t* buf = mybufs + (turn % C::NBUF) * C::BUF;
              ++turn;
              if (issuer) bulk_wait_read<C::NBUF - 1>();   // the buffer's last store has read it
              group_sync(1 + h);
              if (mirror) put_columns(buf, row, w);
              else put_rows(buf, row, w);
              tc::fence_proxy_async();
              group_sync(1 + h);
              if (issuer) {
                if (mirror) tma_store_3d(&g.maps[q][1 + 3 * part], buf, 0, c0, r0 / 64);
                else tma_store_2d(&g.maps[q][2 + 3 * part], buf, c0, r0);
                bulk_commit();
              }
            }
          }
        }
      }
      if constexpr (!kFull) ++gsub;
    }
    if (issuer) bulk_wait();   // written before the next launch reads
  }
  tc::tc_fence_before();
  __syncwarp();
  tc::cluster_sync();   // every MMA of the pair has completed; no peer arrival is pending
  if (warp == 1) tc::tmem_dealloc_pair(tmem, 512);
}

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

// A call's polynomial: coefficients and the powers of two that the matrices are stored with.
struct Plan {
  int steps = 0;
  double a[kMaxSteps], b[kMaxSteps], c[kMaxSteps];
  double sx[kMaxSteps + 1], sl[kMaxSteps], sm[kMaxSteps];   // of X_k, L and M of step k
};
double below_2_15(double bound) { return std::exp2(std::floor(std::log2(32000.0 / bound))); }
kfac_status make_plan(const kfac_ortho_desc* d, Plan* p) {
  p->steps = d->steps;
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
    double next = std::sqrt(u * u) * poly(u * u);
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
    p->sx[k] = k == 0 ? 1.0 : below_2_15(u);   // X_0's factor is r, on the device
    p->sl[k] = below_2_15(u * u);
    p->sm[k] = below_2_15(v);
    u = next;
  }
  p->sx[d->steps] = 1.0;
  return KFAC_OK;
}

struct Matrix {
  int rows, cols, s, l, tall, xp, sp;    // pitches of X and of the s x s matrices
  size_t x[2][2], gram[2], poly[2], part, r;   // [buffer][hi, lo]
  int prep_blocks, tx;
};
int64_t pitch_of(int64_t cols) { return cdiv(cols, 64) * 64; }

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

// Regions of the workspace; matrices without elements take none and are left out.
size_t lay_out(const kfac_ortho_desc* d, int count, const int* rows, const int* cols,
               std::vector<Matrix>* out) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes);
    return here;
  };
  const int halves = d->math == KFAC_ORTHO_FULL ? 2 : 1;
  for (int i = 0; i < count; ++i) {
    Matrix m{};
    m.rows = rows[i];
    m.cols = cols[i];
    m.s = std::min(rows[i], cols[i]);
    m.l = std::max(rows[i], cols[i]);
    m.tall = rows[i] > cols[i];
    if (m.s > 0) {
      m.xp = (int)pitch_of(m.cols);
      m.sp = (int)pitch_of(m.s);
      for (int b = 0; b < (d->steps > 1 ? 2 : 1); ++b)
        for (int h = 0; h < halves; ++h) m.x[b][h] = take((size_t)m.rows * m.xp * 2);
      for (int h = 0; h < halves; ++h) {
        m.gram[h] = take((size_t)m.s * m.sp * 2);
        m.poly[h] = take((size_t)m.s * m.sp * 2);
      }
      m.part = take(kPrepBlocks * 3 * sizeof(float));
      m.r = take(sizeof(float));
    }
    if (out) out->push_back(m);
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

template <int PH, typename TO, bool kFull>
kfac_status launch_product(const Launch<kFull>& g, cudaStream_t st) {
  using C = Cfg<kFull>;
  static OncePerDevice once;
  if (kfac_status e = allow_smem(once, ortho_product_kernel<PH, TO, kFull>, C::SMEM)) return e;
  const int pairs = std::max(1, std::min(g.tile_start[g.count], num_sms() / 2));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, ortho_product_kernel<PH, TO, kFull>, g);
  count_launch();
  return check_launch();
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

// The matrices of `idx` (at most kMaxGroup, none empty), all launches.
template <bool kFull>
kfac_status run_group(const Call& c, const Plan& plan, const std::vector<Matrix>& ms,
                      const std::vector<int>& idx, char* ws, cudaStream_t st) {
  const int n = (int)idx.size();
  const int halves = kFull ? 2 : 1;
  auto half_at = [&](size_t off) { return reinterpret_cast<__half*>(ws + off); };
  const bool bf16 = c.d->dtype == KFAC_BF16;
  const size_t es = bf16 ? 2 : 4;
  {
    std::unique_ptr<PrepLaunch> g(new PrepLaunch());
    int blocks = 0;
    for (int i = 0; i < n; ++i) {
      const Matrix& m = ms[idx[i]];
      PrepTask& t = g->task[i];
      t.x = c.x[idx[i]];
      t.ldx = c.ldx[idx[i]];
      t.m = c.hp ? c.momentum[idx[i]] : nullptr;
      t.ldm = c.hp ? c.ldm[idx[i]] : 0;
      t.hi = half_at(m.x[0][0]);
      t.lo = kFull ? half_at(m.x[0][1]) : nullptr;
      t.part = reinterpret_cast<float*>(ws + m.part);
      t.r = reinterpret_cast<float*>(ws + m.r);
      t.rows = m.rows;
      t.cols = m.cols;
      t.pitch = m.xp;
      const int vn = 16 / (int)es;
      t.vec = m.cols % vn == 0 && (uintptr_t)t.x % 16 == 0 && (m.rows == 1 || t.ldx % vn == 0) &&
              (!c.hp || ((uintptr_t)t.m % 16 == 0 && (m.rows == 1 || t.ldm % 4 == 0)));
      const int pieces = (int)cdiv(m.cols, t.vec ? vn : 1);
      t.tx = 1;
      while (t.tx < pieces && t.tx < kPrepThreads) t.tx *= 2;
      g->block_start[i] = blocks;
      // a few pieces per thread; one wave of the largest matrices
      const int64_t rpb = kPrepThreads / t.tx, per = cdiv(pieces, t.tx);
      blocks += (int)std::max<int64_t>(1, std::min<int64_t>(kPrepBlocks, cdiv((int64_t)m.rows * per, rpb * 4)));
    }
    g->block_start[n] = blocks;
    g->count = n;
    g->mu = c.hp ? (float)c.hp->momentum : 0.f;
    g->nesterov = c.hp ? c.hp->nesterov : 0;
    g->eps = (float)c.d->eps;
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
  // every matrix's maps, once: X (two buffers) and the s x s matrices, in both kinds of boxes
  struct Maps {
    CUtensorMap x[2][2][2], gram[2][2], poly[2][2];   // [buffer][hi, lo][rows, chunks]
  };
  std::vector<Maps> maps(n);
  for (int i = 0; i < n; ++i) {
    const Matrix& m = ms[idx[i]];
    for (int h = 0; h < halves; ++h) {
      for (int k = 0; k < 2; ++k) {
        for (int b = 0; b < (plan.steps > 1 ? 2 : 1); ++b)
          if (!make_map(&maps[i].x[b][h][k], half_at(m.x[b][h]), m.rows, m.cols, m.xp, k)) return KFAC_ERR_CUDA;
        if (!make_map(&maps[i].gram[h][k], half_at(m.gram[h]), m.s, m.s, m.sp, k) ||
            !make_map(&maps[i].poly[h][k], half_at(m.poly[h]), m.s, m.s, m.sp, k))
          return KFAC_ERR_CUDA;
      }
    }
  }
  std::unique_ptr<Launch<kFull>> g(new Launch<kFull>());
  for (int step = 0; step < plan.steps; ++step) {
    const int cur = step & 1;
    const bool last = step + 1 == plan.steps;
    for (int ph = 0; ph < 3; ++ph) {
      int tiles = 0;
      for (int i = 0; i < n; ++i) {
        const Matrix& m = ms[idx[i]];
        Task& t = g->task[i];
        t = Task{};
        t.r = reinterpret_cast<const float*>(ws + m.r);
        const double sx = plan.sx[step], sl = plan.sl[step], sm = plan.sm[step];
        for (int h = 0; h < halves; ++h) {
          CUtensorMap* to = &g->maps[i][3 * h];
          if (ph == 0) {
            to[0] = maps[i].x[cur][h][m.tall];
            to[1] = maps[i].gram[h][1];
            to[2] = maps[i].gram[h][0];
          } else if (ph == 1) {
            to[0] = maps[i].gram[h][0];
            to[1] = maps[i].poly[h][1];
            to[2] = maps[i].poly[h][0];
          } else {
            to[0] = m.tall ? maps[i].x[cur][h][0] : maps[i].poly[h][0];
            to[1] = m.tall ? maps[i].poly[h][0] : maps[i].x[cur][h][1];
            if (!last) to[2] = maps[i].x[cur ^ 1][h][0];
          }
        }
        if (ph == 0) {
          t.M = t.N = m.s;
          t.kblocks = (int)cdiv(m.l, 64);
          t.mn_a = t.mn_b = m.tall;
          t.alpha = (float)(sl / (sx * sx));
          t.rpow = step == 0 ? 2 : 0;
        } else if (ph == 1) {
          t.M = t.N = m.s;
          t.kblocks = (int)cdiv(m.s, 64);
          t.alpha = (float)(sm * plan.c[step] / (sl * sl));
          t.beta = (float)(sm * plan.b[step] / sl);
          t.diag = (float)(sm * plan.a[step]);
          t.add_hi = half_at(m.gram[0]);
          t.add_lo = kFull ? half_at(m.gram[1]) : nullptr;
          t.add_pitch = m.sp;
        } else {
          t.M = m.rows;
          t.N = m.cols;
          t.kblocks = (int)cdiv(m.s, 64);
          t.mn_b = !m.tall;
          t.alpha = (float)(plan.sx[step + 1] / (sm * sx));
          t.rpow = step == 0 ? 1 : 0;
          if (last) {
            t.out = c.out[idx[i]];
            t.out_ld = c.ldo[idx[i]];
            if (c.hp) {
              t.keep = (float)(1.0 - c.hp->lr * c.hp->weight_decay);
              t.rate = (float)(c.hp->lr * c.hp->update_scale *
                               std::sqrt(std::max(1.0, (double)m.rows / (double)m.cols)));
            }
          }
        }
        t.upper = ph < 2;
        t.tiles_m = (int)cdiv(t.M, 256);
        t.tiles_n = (int)cdiv(t.N, 256);
        g->tile_start[i] = tiles;
        tiles += t.upper ? t.tiles_m * (t.tiles_m + 1) / 2 : t.tiles_m * t.tiles_n;
      }
      g->tile_start[n] = tiles;
      g->count = n;
      kfac_status e;
      if (ph == 0) e = launch_product<PH_GRAM, float, kFull>(*g, st);
      else if (ph == 1) e = launch_product<PH_POLY, float, kFull>(*g, st);
      else if (!last) e = launch_product<PH_APPLY, float, kFull>(*g, st);
      else if (c.hp) e = launch_product<PH_STEP, float, kFull>(*g, st);
      else if (bf16) e = launch_product<PH_OUT, __nv_bfloat16, kFull>(*g, st);
      else e = launch_product<PH_OUT, float, kFull>(*g, st);
      if (e) return e;
    }
  }
  return KFAC_OK;
}

kfac_status run(const Call& c, int count, const int* rows, const int* cols, void* workspace,
                size_t bytes, cudaStream_t st) {
  Plan plan;
  if (kfac_status e = make_plan(c.d, &plan)) return e;
  std::vector<Matrix> ms;
  const size_t need = lay_out(c.d, count, rows, cols, &ms);
  if (need && (!workspace || (uintptr_t)workspace % kAlign || bytes < need)) return KFAC_ERR_WORKSPACE;
  // longest reductions first: the last round of tiles then holds the shortest
  std::vector<int> order;
  for (int i = 0; i < count; ++i)
    if (ms[i].s > 0) order.push_back(i);
  std::stable_sort(order.begin(), order.end(), [&](int a, int b) { return ms[a].l > ms[b].l; });
  for (size_t at = 0; at < order.size(); at += kMaxGroup) {
    const std::vector<int> idx(order.begin() + at, order.begin() + std::min(order.size(), at + kMaxGroup));
    kfac_status e = c.d->math == KFAC_ORTHO_FULL
                        ? run_group<true>(c, plan, ms, idx, static_cast<char*>(workspace), st)
                        : run_group<false>(c, plan, ms, idx, static_cast<char*>(workspace), st);
    if (e) return e;
  }
  return KFAC_OK;
}

bool bad_matrix(const void* p, int64_t ld, int rows, int cols, size_t es) {
  return !p || (uintptr_t)p % es || ld < 0 || ld > (int64_t(1) << 40) || (rows > 1 && ld < cols);
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
  *bytes = lay_out(d, count, rows, cols, nullptr);
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
  return guarded([&] { return run(c, count, rows, cols, workspace, workspace_bytes, stream); });
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
  for (int i = 0; i < count; ++i) {
    if (rows[i] == 0 || cols[i] == 0) continue;
    if (bad_matrix(grad[i], ldg[i], rows[i], cols[i], es) ||
        bad_matrix(momentum[i], ldm[i], rows[i], cols[i], 4) ||
        bad_matrix(param[i], ldp[i], rows[i], cols[i], 4))
      return KFAC_ERR_INVALID_ARG;
  }
  return guarded([&] {
    std::vector<void*> out(param, param + count);
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
