// Dropout with the residual added, its mask from a counter-based generator:
//   u_i = word i mod 4 of Philox4x32-10(counter = (i / 4, offset), key = seed)
//   y_i = r_i + (u_i >= floor(p 2^32) ? x_i / (1 - p) : 0),  i the row-major index.
// The backward pass is the same function of the output gradient without r: the mask
// is generated again from (seed, offset) and never stored.
//
// Philox4x32-10: Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as
// 1, 2, 3" (SC 2011): ten rounds of two 32 x 32 -> 64 bit products.  A thread takes two
// 16-byte vectors of x: one generator block per four elements.  Bound by memory with a
// residual or in fp32 (16384 x 2048 bf16 with residual, 201 MB: 30.6 us, 6.6 TB/s; one
// vector per thread took 35 us, four 33.5), by the generator without one in bf16 (16 bytes
// per generator block: 30 us, 4.5 TB/s).  Sums in fp32, one rounding at the store.  A
// dropped x is not multiplied, so an infinity or NaN there does not reach y.
#include "kfac_internal.cuh"

#include <cmath>

namespace kfac {
namespace {

constexpr int kDropThreads = 256;
constexpr int kVecs = 2;         // 16-byte vectors per thread, a block's width apart

struct DropArgs {
  const void *x, *r;
  void* y;
  int64_t n;                    // rows * cols
  int64_t cols, ldx, ldr, ldy;
  uint32_t seed_lo, seed_hi, off_lo, off_hi;
  uint32_t threshold;           // below it: dropped
  bool all;                     // p = 1: everything is
  float scale;
};

__device__ __forceinline__ uint4 philox(uint64_t block, const DropArgs& a) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = a.off_lo, c3 = a.off_hi;
  uint32_t k0 = a.seed_lo, k1 = a.seed_hi;
#pragma unroll
  for (int round = 0; round < 10; ++round) {
    const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ float drop1(float x, float r, uint32_t u, const DropArgs& a) {
  return r + (u >= a.threshold && !a.all ? x * a.scale : 0.f);
}

template <typename T> struct alignas(16) Pack { T v[16 / sizeof(T)]; };

// x, r, y contiguous and 16-byte aligned; the last threads' element by element.
template <typename T, bool kRes>
__global__ void __launch_bounds__(kDropThreads) dropout_flat_kernel(const __grid_constant__ DropArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int N = 16 / (int)sizeof(T);
  const T* x = static_cast<const T*>(a.x);
  const T* r = static_cast<const T*>(a.r);
  T* y = static_cast<T*>(a.y);
  const int64_t first = ((int64_t)blockIdx.x * kDropThreads * kVecs + threadIdx.x) * N;
  if (first + (int64_t)(kVecs - 1) * kDropThreads * N + N <= a.n) {   // all of them whole
    Pack<T> px[kVecs], pr[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int64_t i = first + (int64_t)v * kDropThreads * N;
      px[v] = *reinterpret_cast<const Pack<T>*>(x + i);
      if (kRes) pr[v] = *reinterpret_cast<const Pack<T>*>(r + i);
    }
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int64_t i = first + (int64_t)v * kDropThreads * N;
      Pack<T> py;
#pragma unroll
      for (int b = 0; b < N / 4; ++b) {
        const uint4 u = philox((uint64_t)(i / 4 + b), a);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          py.v[4 * b + j] = (T)drop1(to_f32<T>(px[v].v[4 * b + j]),
                                     kRes ? to_f32<T>(pr[v].v[4 * b + j]) : 0.f, w[j], a);
      }
      *reinterpret_cast<Pack<T>*>(y + i) = py;
    }
    return;
  }
  for (int v = 0; v < kVecs; ++v) {
    const int64_t i = first + (int64_t)v * kDropThreads * N;
    for (int b = 0; b < N / 4 && i < a.n; ++b) {
      const uint4 u = philox((uint64_t)(i / 4 + b), a);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      for (int j = 0; j < 4; ++j) {
        const int64_t e = i + 4 * b + j;
        if (e < a.n) y[e] = (T)drop1(to_f32<T>(x[e]), kRes ? to_f32<T>(r[e]) : 0.f, w[j], a);
      }
    }
  }
}

// Any leading dimensions and alignment: one generator block (four elements of the
// row-major index) per thread, element by element.  Bound by its loads and stores of single
// elements (16384 x 2047 with residual, bf16 85 us, fp32 91 us; without 73 and 78 us).
template <typename T, bool kRes>
__global__ void __launch_bounds__(kDropThreads) dropout_strided_kernel(const __grid_constant__ DropArgs a) {
  pdl_wait();
  pdl_trigger();
  const T* x = static_cast<const T*>(a.x);
  const T* r = static_cast<const T*>(a.r);
  T* y = static_cast<T*>(a.y);
  const int64_t i = ((int64_t)blockIdx.x * kDropThreads + threadIdx.x) * 4;
  if (i >= a.n) return;
  const uint4 u = philox((uint64_t)(i / 4), a);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  int64_t row = i / a.cols, col = i - row * a.cols;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (i + j < a.n) {
      y[row * a.ldy + col] = (T)drop1(to_f32<T>(x[row * a.ldx + col]),
                                      kRes ? to_f32<T>(r[row * a.ldr + col]) : 0.f, w[j], a);
      if (++col == a.cols) {
        col = 0;
        ++row;
      }
    }
  }
}

template <typename T>
void launch_dropout(const DropArgs& a, bool flat, cudaStream_t st) {
  const int64_t per = flat ? 16 / (int64_t)sizeof(T) * kVecs : 4;
  const dim3 grid((unsigned)cdiv(cdiv(a.n, per), kDropThreads)), block(kDropThreads);
  if (flat) {
    if (a.r) launch_pdl(dropout_flat_kernel<T, true>, grid, block, 0, st, a);
    else launch_pdl(dropout_flat_kernel<T, false>, grid, block, 0, st, a);
  } else {
    if (a.r) launch_pdl(dropout_strided_kernel<T, true>, grid, block, 0, st, a);
    else launch_pdl(dropout_strided_kernel<T, false>, grid, block, 0, st, a);
  }
}

}  // namespace
}  // namespace kfac

using namespace kfac;

extern "C" kfac_status kfac_dropout(int dtype, const void* x, int64_t ldx, const void* residual,
                                    int64_t ldr, void* out, int64_t ldo, int64_t rows,
                                    int64_t cols, double p, uint64_t seed, uint64_t offset,
                                    cudaStream_t stream) {
  if (dtype != KFAC_F32 && dtype != KFAC_BF16) return KFAC_ERR_INVALID_ARG;
  if (!(p >= 0.0 && p <= 1.0) || rows < 0 || cols < 0) return KFAC_ERR_INVALID_ARG;
  if (rows > 0 && cols > (int64_t(1) << 40) / rows) return KFAC_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return KFAC_OK;
  const size_t es = dtype == KFAC_BF16 ? 2 : 4;
  auto bad = [&](const void* q, int64_t ld) {
    return (uintptr_t)q % es || ld < 0 || (rows > 1 && ld < cols);
  };
  if (!x || !out || bad(x, ldx) || bad(out, ldo) || (residual && bad(residual, ldr)))
    return KFAC_ERR_INVALID_ARG;
  DropArgs a{};
  a.x = x;
  a.r = residual;
  a.y = out;
  a.n = rows * cols;
  a.cols = cols;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldy = ldo;
  a.seed_lo = (uint32_t)seed;
  a.seed_hi = (uint32_t)(seed >> 32);
  a.off_lo = (uint32_t)offset;
  a.off_hi = (uint32_t)(offset >> 32);
  a.all = p >= 1.0;
  a.threshold = a.all ? 0u : (uint32_t)std::floor(p * 4294967296.0);
  a.scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f;
  auto dense = [&](const void* q, int64_t ld) {
    return !q || ((uintptr_t)q % 16 == 0 && (rows == 1 || ld == cols));
  };
  const bool flat = dense(x, ldx) && dense(residual, ldr) && dense(out, ldo);
  if (dtype == KFAC_BF16) launch_dropout<__nv_bfloat16>(a, flat, stream);
  else launch_dropout<float>(a, flat, stream);
  count_launch();
  return check_launch();
}
