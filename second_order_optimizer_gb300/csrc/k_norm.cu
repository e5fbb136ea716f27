// Root-mean-square norm with the residual's addition, an 8-bit output, and the gradients:
//   s = x + residual,  r = (mean_j s_j^2 + eps)^(-1/2),  h = s,  y = s r gain,
//   q = e4m3(y / scale), scale = max |y| / 448 over a group of channels;
//   n = h r,  w = dy gain,  dx = r (w - n mean_j(w_j n_j)) + dh,
//   dgain_j = sum_rows dy_j n_j,  dgain_square_j = mean_rows (dy_j n_j)^2.
//
// Bound by memory: each tensor crosses it once.  A row stays in the registers of the threads
// that share it (a warp, 256 or 1024 threads) between its sum and its use, in vectors of 16
// bytes where rows and columns allow, else in pairs or element by element; rows wider than that
// are read again (from L2).  Statistics, sums and products in fp32, one rounding at each store.
//
// The gradients of the gain sum over the rows.  A block walks rows a grid apart and keeps its
// threads' columns in registers; its sums go to the workspace and a second launch adds the
// blocks' in order, so that no atomics are needed and the same inputs give the same bits.
#include "kfac_internal.cuh"
#include "per_device.h"

#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

namespace kfac {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr int64_t kMaxCols = 1 << 20;
constexpr int kMaxGroups = 8192;   // of a row's 8-bit output: their maxima are in shared memory

struct NormArgs {
  const void *x, *r;
  const float* gain;
  void *h, *y;
  float* rstd;
  uint8_t* q;
  float* scales;
  int64_t rows, ldx, ldr, ldh, ldy, ldq;
  int cols, group, groups;
  int shift;               // channel >> shift: its group (31: one for the row)
  float inv_cols, eps;
};

template <typename T, int N> struct alignas(N * sizeof(T)) Vec { T v[N]; };

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the TPR threads of a row; every thread gets it.  red: a float per warp and slot
// of the block, the slot another than in the call before.
template <int TPR> __device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    constexpr int W = TPR / 32;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = lane < W ? red[lane] : 0.f;
    v = warp_sum(v);
  }
  return v;
}

// gain[c .. c + N), ones where there is none (N > 1: 4 N bytes aligned, at most 16).
template <int N>
__device__ __forceinline__ void load_gain(const float* gain, int c, int cols, float (&g)[N]) {
  if (!gain || c >= cols) {
#pragma unroll
    for (int i = 0; i < N; ++i) g[i] = 1.f;
  } else if constexpr (N == 1) {
    g[0] = __ldg(gain + c);
  } else if constexpr (N == 2) {
    *reinterpret_cast<float2*>(&g[0]) = __ldg(reinterpret_cast<const float2*>(gain + c));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(&g[i]) = __ldg(reinterpret_cast<const float4*>(gain + c + i));
  }
}

// |v| as an integer: ordered like the values, NaN above infinity.
__device__ __forceinline__ int abs_bits(float v) { return __float_as_int(v) & 0x7fffffff; }

// N values over their group's scale as e4m3 (two per conversion).
template <int N>
__device__ __forceinline__ void e4m3_of(const float (&v)[N], float scale, Vec<uint8_t, N>& q) {
  float u[N];
#pragma unroll
  for (int i = 0; i < N; ++i) u[i] = scale == 0.f ? 0.f : v[i] / scale;
  if constexpr (N == 1) {
    q.v[0] = (uint8_t)__nv_cvt_float_to_fp8(u[0], __NV_SATFINITE, __NV_E4M3);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const __nv_fp8x2_storage_t two =
          __nv_cvt_float2_to_fp8x2(make_float2(u[i], u[i + 1]), __NV_SATFINITE, __NV_E4M3);
      q.v[i] = (uint8_t)(two & 0xff);
      q.v[i + 1] = (uint8_t)(two >> 8);
    }
  }
}

// A row per TPR threads, all of it in registers: thread t holds vectors t, t + TPR, ... of N
// elements.  kQuant: with the 8-bit output; the groups' maxima meet in shared memory (a
// maximum is the same in any order).
template <typename T, int N, int TPR, int V, bool kRes, bool kQuant>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256)
    norm_rows_kernel(const __grid_constant__ NormArgs a) {
  constexpr int BLOCK = TPR > 256 ? TPR : 256, RPB = BLOCK / TPR;
  extern __shared__ int amax[];   // kQuant: [RPB][groups]
  __shared__ float red[32];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + sub;
  const bool live = row < a.rows;
  pdl_wait();
  pdl_trigger();
  using Pack = Vec<T, N>;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* r = static_cast<const T*>(a.r) + row * a.ldr;
  float s[V][N], gain[V][N];
  float sum = 0.f;
  if (live) {
    Pack px[V], pr[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * TPR + t) * N;
      if (c < a.cols) {
        px[v] = *reinterpret_cast<const Pack*>(x + c);
        if (kRes) pr[v] = *reinterpret_cast<const Pack*>(r + c);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) load_gain<N>(a.gain, (v * TPR + t) * N, a.cols, gain[v]);
    T* h = static_cast<T*>(a.h) + row * a.ldh;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * TPR + t) * N;
      if (c < a.cols) {
        Pack ph;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          s[v][i] = to_f32<T>(px[v].v[i]);
          if (kRes) s[v][i] += to_f32<T>(pr[v].v[i]);
          ph.v[i] = (T)s[v][i];
          sum = fmaf(s[v][i], s[v][i], sum);
        }
        if (a.h) *reinterpret_cast<Pack*>(h + c) = ph;
      }
    }
  }
  if (kQuant) {
    for (int g = threadIdx.x; g < RPB * a.groups; g += BLOCK) amax[g] = 0;
    if (TPR == 32) __syncthreads();   // otherwise the one inside row_sum
  }
  sum = row_sum<TPR>(sum, red);
  const float rstd = rsqrtf(fmaf(sum, a.inv_cols, a.eps));
  if (live && t == 0 && a.rstd) a.rstd[row] = rstd;
  T* y = static_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * TPR + t) * N;
    if (live && c < a.cols) {
      Pack py;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        s[v][i] = s[v][i] * rstd * gain[v][i];
        py.v[i] = (T)s[v][i];
      }
      if (a.y) *reinterpret_cast<Pack*>(y + c) = py;
    }
  }
  if constexpr (kQuant) {
    // a group's channels lie beside each other: its maximum is that of some neighbouring lanes, or of
    // whole warps
    const int lanes = a.group == 0 ? 32 : min(32, a.group / N);
    int top[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      top[v] = 0;
      if (live && (v * TPR + t) * N < a.cols) {
#pragma unroll
        for (int i = 0; i < N; ++i) top[v] = max(top[v], abs_bits(s[v][i]));
      }
      for (int o = lanes / 2; o > 0; o >>= 1) top[v] = max(top[v], __shfl_xor_sync(0xffffffffu, top[v], o));
    }
    if (a.group == 0 || a.group / N > 32) {   // the warps' maxima meet in shared memory
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * TPR + t) * N;
        if (threadIdx.x % 32 == 0 && live && c < a.cols)
          atomicMax(&amax[sub * a.groups + (c >> a.shift)], top[v]);
      }
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * TPR + t) * N;
        if (c < a.cols) top[v] = amax[sub * a.groups + (c >> a.shift)];
      }
    }
    uint8_t* q = a.q + row * a.ldq;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * TPR + t) * N;
      if (live && c < a.cols) {
        const float scale = __int_as_float(top[v]) / kE4m3Max;
        if (c == (c >> a.shift) << a.shift)   // the group's first channels
          a.scales[row * a.groups + (c >> a.shift)] = scale;
        Vec<uint8_t, N> pq;
        e4m3_of<N>(s[v], scale, pq);
        *reinterpret_cast<Vec<uint8_t, N>*>(q + c) = pq;
      }
    }
  }
}

// A row of any width per block, read twice (three times with the 8-bit output).
template <typename T>
__global__ void __launch_bounds__(1024) norm_wide_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ int amax[];
  __shared__ float red[32];
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* r = a.r ? static_cast<const T*>(a.r) + row * a.ldr : nullptr;
  // h may be x or residual: what is read again after it was written there comes from it
  T* h = a.h ? static_cast<T*>(a.h) + row * a.ldh : nullptr;
  T* y = a.y ? static_cast<T*>(a.y) + row * a.ldy : nullptr;
  auto at = [&](int c) { return to_f32<T>(x[c]) + (r ? to_f32<T>(r[c]) : 0.f); };
  float sum = 0.f;
  for (int c = threadIdx.x; c < a.cols; c += 1024) {
    const float s = at(c);
    sum = fmaf(s, s, sum);
  }
  if (a.q)
    for (int g = threadIdx.x; g < a.groups; g += 1024) amax[g] = 0;
  sum = row_sum<1024>(sum, red);
  const float rstd = rsqrtf(fmaf(sum, a.inv_cols, a.eps));
  if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
  auto norm = [&](int c, float s) { return s * rstd * (a.gain ? __ldg(a.gain + c) : 1.f); };
  if (a.q) {
    for (int c = threadIdx.x; c < a.cols; c += 1024)
      atomicMax(&amax[c >> a.shift], abs_bits(norm(c, at(c))));
    __syncthreads();
    for (int g = threadIdx.x; g < a.groups; g += 1024)
      a.scales[row * a.groups + g] = __int_as_float(amax[g]) / kE4m3Max;
  }
  for (int c = threadIdx.x; c < a.cols; c += 1024) {   // each element by one thread: h in place
    const float s = at(c), v = norm(c, s);
    if (h) h[c] = (T)s;
    if (y) y[c] = (T)v;
    if (a.q) {
      const float one[1] = {v};
      Vec<uint8_t, 1> pq;
      e4m3_of<1>(one, __int_as_float(amax[c >> a.shift]) / kE4m3Max, pq);
      a.q[row * a.ldq + c] = pq.v[0];
    }
  }
}

template <typename T, int N, int TPR, int V>
void launch_norm_rows(const NormArgs& a, cudaStream_t st) {
  constexpr int BLOCK = TPR > 256 ? TPR : 256, RPB = BLOCK / TPR;
  const dim3 grid((unsigned)cdiv(a.rows, RPB)), block(BLOCK);
  if (a.q) {
    const size_t smem = (size_t)RPB * a.groups * sizeof(int);
    if (a.r) launch_pdl(norm_rows_kernel<T, N, TPR, V, true, true>, grid, block, smem, st, a);
    else launch_pdl(norm_rows_kernel<T, N, TPR, V, false, true>, grid, block, smem, st, a);
  } else {
    if (a.r) launch_pdl(norm_rows_kernel<T, N, TPR, V, true, false>, grid, block, 0, st, a);
    else launch_pdl(norm_rows_kernel<T, N, TPR, V, false, false>, grid, block, 0, st, a);
  }
}

// Threads per row: 256 with as many vectors each as the row needs; a warp for narrow rows (single
// elements too: 16384 x 199 in bf16 8.3 us, 256 threads 20.6); 1024 for wide ones.  Pairs of elements
// where rows are no whole vectors but even: 16384 x 1002, fp32 with the 8-bit output 53 us for 82, bf16
// 55 for 82, without it 29 for 37.  (4096 x 8190 with the 8-bit output: fp32 256 threads 232 us,
// 1024 134; bf16 without it 256 threads 49, 1024 83.)
template <typename T, int N> bool launch_norm(const NormArgs& a, cudaStream_t st) {
  constexpr bool kWhole = N * sizeof(T) == 16;
  const int64_t vecs = cdiv(a.cols, N);
  if (vecs <= 32) launch_norm_rows<T, N, 32, 1>(a, st);
  else if (vecs <= 64) launch_norm_rows<T, N, 32, 2>(a, st);
  else if constexpr (kWhole) {
    if (vecs <= 256) launch_norm_rows<T, N, 256, 1>(a, st);
    else if (vecs <= 512) launch_norm_rows<T, N, 256, 2>(a, st);
    else if (vecs <= 1024) launch_norm_rows<T, N, 256, 4>(a, st);
    else if (vecs <= 2048) launch_norm_rows<T, N, 1024, 2>(a, st);
    else return false;
  } else {
    if (N == 2 && vecs <= 128) launch_norm_rows<T, 2, 32, 4>(a, st);
    else if (vecs <= 256) launch_norm_rows<T, N, 32, 8>(a, st);
    else if (vecs <= 512) launch_norm_rows<T, N, 256, 2>(a, st);
    else if (vecs <= 1024) launch_norm_rows<T, N, 256, 4>(a, st);
    else if (vecs <= 2048) launch_norm_rows<T, N, 256, 8>(a, st);
    else if (N == 2 && sizeof(T) == 4 && vecs <= 4096) launch_norm_rows<float, 2, 1024, 4>(a, st);
    else if (vecs <= 4096) launch_norm_rows<T, N, 256, 16>(a, st);
    else if (N == 1 && vecs <= 8192) launch_norm_rows<T, 1, 1024, 8>(a, st);
    else return false;
  }
  return true;
}

// ------------------------------------------------------------------------------ backward

struct NormGradArgs {
  const void *dy, *h, *dh;
  const float *gain, *rstd;
  void* dx;
  float *part;            // [parts][2][cols]
  float *dgain, *dgain_sq;
  int64_t rows, lddy, ldh, lddh, lddx;
  int cols, parts;
  float inv_cols, inv_rows;
};

// Rows a grid apart, R at a time, TPR threads each; thread t holds vectors t, t + TPR, ...
// Each thread copies what it will use itself into a ring of its own in shared memory (cp.async,
// STAGES - 1 rounds of R rows ahead), so that loads stay in flight through the sums and stores and no
// barrier orders the ring.  Single bf16 elements are below cp.async's 4 bytes: they are loaded
// when they are used.  Of 16384 x 2048 (bf16, 268 MB) loads of four rows at a time into registers
// took 111 us; rounds of two rows from the ring 58, of three 46.
template <typename T, int N, int TPR, int V, int R, bool kDh> struct GradRing {
  static constexpr bool kOn = N * sizeof(T) >= 4;
  static constexpr int BLOCK = TPR > 256 ? TPR : 256, TENSORS = kDh ? 3 : 2;
  static constexpr size_t ROUND = (size_t)R * TENSORS * V * BLOCK * N * sizeof(T);
  // room for two blocks an SM (less than whole vectors: four, see backward_parts)
  static constexpr int STAGES = N * sizeof(T) < 16 ? 2 : ROUND * 4 <= 112 * 1024 ? 4 : ROUND * 3 <= 112 * 1024 ? 3 : 2;
  static_assert(STAGES * ROUND <= 220 * 1024, "shared memory");
  static constexpr size_t BYTES = kOn ? STAGES * ROUND : 0;
};
template <int BYTES> __device__ __forceinline__ void copy_async(void* dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

template <typename T, int N, int TPR, int V, int R, bool kDh>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256)
    norm_backward_kernel(const __grid_constant__ NormGradArgs a) {
  using Ring = GradRing<T, N, TPR, V, R, kDh>;
  constexpr int BLOCK = Ring::BLOCK, RPB = BLOCK / TPR, W = TPR / 32, TENSORS = Ring::TENSORS;
  constexpr int STAGES = Ring::STAGES;
  extern __shared__ __align__(16) uint8_t shared[];   // the ring; then, TPR == 32: [RPB][2][32 V N]
  __shared__ float red[2][R][32];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  using Pack = Vec<T, N>;
  Pack* ring = reinterpret_cast<Pack*>(shared);
  pdl_wait();
  pdl_trigger();
  float gain[V][N], dg[V][N], sq[V][N];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    load_gain<N>(a.gain, (v * TPR + t) * N, a.cols, gain[v]);
#pragma unroll
    for (int i = 0; i < N; ++i) dg[v][i] = sq[v][i] = 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * RPB;
  const int64_t first = (int64_t)blockIdx.x * RPB + sub;
  const int rounds = (int)((a.rows - (int64_t)blockIdx.x * RPB + R * step - 1) / (R * step));
  const T* src[TENSORS] = {static_cast<const T*>(a.dy), static_cast<const T*>(a.h)};
  int64_t ld[TENSORS] = {a.lddy, a.ldh};
  if constexpr (kDh) {
    src[2] = static_cast<const T*>(a.dh);
    ld[2] = a.lddh;
  }
  auto slot = [&](int round, int j, int k, int v) {
    return ring + ((((round % STAGES) * R + j) * TENSORS + k) * V + v) * BLOCK + threadIdx.x;
  };
  auto fetch = [&](int round) {   // always a group, so that the waits count rounds
    if constexpr (Ring::kOn) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int64_t row = first + ((int64_t)round * R + j) * step;
        if (round < rounds && row < a.rows) {
#pragma unroll
          for (int k = 0; k < TENSORS; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
              const int c = (v * TPR + t) * N;
              if (c < a.cols) copy_async<N * sizeof(T)>(slot(round, j, k, v), src[k] + row * ld[k] + c);
            }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(s);
  for (int round = 0; round < rounds; ++round) {
    const int turn = round & 1;
    const int64_t row0 = first + (int64_t)round * R * step;
    Pack pg[R][V], ph[R][V], pd[R][V];
    float rstd[R];
#pragma unroll
    for (int j = 0; j < R; ++j)
      rstd[j] = row0 + j * step < a.rows ? __ldg(a.rstd + row0 + j * step) : 0.f;
    if constexpr (Ring::kOn) asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t row = row0 + j * step;
      if (row >= a.rows) continue;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * TPR + t) * N;
        if (c >= a.cols) continue;
        if constexpr (Ring::kOn) {
          pg[j][v] = *slot(round, j, 0, v);
          ph[j][v] = *slot(round, j, 1, v);
          if constexpr (kDh) pd[j][v] = *slot(round, j, 2, v);
        } else {
          pg[j][v] = *reinterpret_cast<const Pack*>(src[0] + row * ld[0] + c);
          ph[j][v] = *reinterpret_cast<const Pack*>(src[1] + row * ld[1] + c);
          if constexpr (kDh) pd[j][v] = *reinterpret_cast<const Pack*>(src[2] + row * ld[2] + c);
        }
      }
    }
    fetch(round + STAGES - 1);   // into the slots of the round before, which this thread has read
    float dot[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      dot[j] = 0.f;
      if (row0 + j * step >= a.rows) continue;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if ((v * TPR + t) * N >= a.cols) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float n = to_f32<T>(ph[j][v].v[i]) * rstd[j], g = to_f32<T>(pg[j][v].v[i]);
          const float e = g * n;
          dot[j] = fmaf(e, gain[v][i], dot[j]);
          dg[v][i] += e;
          sq[v][i] = fmaf(e, e, sq[v][i]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) dot[j] = warp_sum(dot[j]);
    if constexpr (TPR > 32) {   // two slots in turn: one barrier per round
      if (lane == 0) {
#pragma unroll
        for (int j = 0; j < R; ++j) red[turn][j][warp] = dot[j];
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < R; ++j) {
        float all = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) all += red[turn][j][w];
        dot[j] = all;
      }
    }
    if (a.dx) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int64_t row = row0 + j * step;
        if (row >= a.rows) continue;
        const float mean = dot[j] * a.inv_cols;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int c = (v * TPR + t) * N;
          if (c >= a.cols) continue;
          Pack px;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float n = to_f32<T>(ph[j][v].v[i]) * rstd[j];
            float d = rstd[j] * (to_f32<T>(pg[j][v].v[i]) * gain[v][i] - n * mean);
            if (kDh) d += to_f32<T>(pd[j][v].v[i]);
            px.v[i] = (T)d;
          }
          *reinterpret_cast<Pack*>(static_cast<T*>(a.dx) + row * a.lddx + c) = px;
        }
      }
    }
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.cols;
  if constexpr (RPB > 1) {   // the block's row groups, in order
    constexpr int C = TPR * V * N;
    float* fold = reinterpret_cast<float*>(shared + Ring::BYTES);
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        fold[(sub * 2 + 0) * C + (v * TPR + t) * N + i] = dg[v][i];
        fold[(sub * 2 + 1) * C + (v * TPR + t) * N + i] = sq[v][i];
      }
    }
    __syncthreads();
    for (int k = threadIdx.x; k < 2 * a.cols; k += BLOCK) {
      const int which = k >= a.cols, c = k - which * a.cols;
      float s = 0.f;
      for (int u = 0; u < RPB; ++u) s += fold[(u * 2 + which) * C + c];
      part[k] = s;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * TPR + t) * N;
      if (c >= a.cols) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        part[c + i] = dg[v][i];
        part[a.cols + c + i] = sq[v][i];
      }
    }
  }
}

// Rows too wide for registers: the means first (rows x parts blocks would re-read them), then
// columns by thread over the rows of a part.
template <typename T>
__global__ void __launch_bounds__(1024) norm_wide_dot_kernel(const __grid_constant__ NormGradArgs a,
                                                             float* means) {
  __shared__ float red[32];
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
  const T* h = static_cast<const T*>(a.h) + row * a.ldh;
  const float rstd = a.rstd[row];
  float dot = 0.f;
  for (int c = threadIdx.x; c < a.cols; c += 1024)
    dot = fmaf(to_f32<T>(dy[c]) * (to_f32<T>(h[c]) * rstd), a.gain ? __ldg(a.gain + c) : 1.f, dot);
  dot = row_sum<1024>(dot, red);
  if (threadIdx.x == 0) means[row] = dot * a.inv_cols;
}
template <typename T>
__global__ void __launch_bounds__(256) norm_wide_backward_kernel(const __grid_constant__ NormGradArgs a,
                                                                 const float* means) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.cols) return;
  const float gain = a.gain ? a.gain[c] : 1.f;
  float dg = 0.f, sq = 0.f;
  for (int64_t row = blockIdx.y; row < a.rows; row += a.parts) {
    const float rstd = __ldg(a.rstd + row);
    const float g = to_f32<T>(static_cast<const T*>(a.dy)[row * a.lddy + c]);
    const float n = to_f32<T>(static_cast<const T*>(a.h)[row * a.ldh + c]) * rstd;
    const float e = g * n;
    dg += e;
    sq = fmaf(e, e, sq);
    if (a.dx) {
      float d = rstd * (g * gain - n * means[row]);
      if (a.dh) d += to_f32<T>(static_cast<const T*>(a.dh)[row * a.lddh + c]);
      static_cast<T*>(a.dx)[row * a.lddx + c] = (T)d;
    }
  }
  if (!a.part) return;
  a.part[((int64_t)blockIdx.y * 2) * a.cols + c] = dg;
  a.part[((int64_t)blockIdx.y * 2 + 1) * a.cols + c] = sq;
}

// The parts' sums, in order: a block takes 32 of the 2 cols columns, warp w every 32nd part.
__global__ void __launch_bounds__(1024) norm_parts_kernel(const __grid_constant__ NormGradArgs a) {
  __shared__ float s[32][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int k = blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (k < 2 * a.cols)
#pragma unroll 10
    for (int p = warp; p < a.parts; p += 32) sum += __ldcg(a.part + (int64_t)p * 2 * a.cols + k);
  s[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && k < 2 * a.cols) {
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) sum += s[w][lane];
    if (k < a.cols) {
      if (a.dgain) a.dgain[k] = sum;
    } else if (a.dgain_sq) {
      a.dgain_sq[k - a.cols] = sum * a.inv_rows;
    }
  }
}

// Blocks of the backward pass: two per SM; four where single elements are loaded, whose blocks
// have less in flight (4099 x 1025 in fp32, forward and backward: 27 us, with two 33; 16384 x 2048 in
// bf16: 94 us with two, 102 with four).
int64_t backward_parts(int64_t rows, bool vec) {
  return std::max<int64_t>(1, std::min<int64_t>(rows, (vec ? 2 : 4) * (int64_t)num_sms()));
}

template <typename T, int N, int TPR, int V, int R, bool kDh>
kfac_status launch_backward_kernel(const NormGradArgs& a, cudaStream_t st) {
  using Ring = GradRing<T, N, TPR, V, R, kDh>;
  constexpr int RPB = Ring::BLOCK / TPR;
  constexpr size_t smem = Ring::BYTES + (RPB > 1 ? (size_t)2 * RPB * TPR * V * N * sizeof(float) : 0);
  static OncePerDevice once;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !once(dev, [] {
        return cudaFuncSetAttribute(norm_backward_kernel<T, N, TPR, V, R, kDh>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess;
      })) {
    check_launch();   // keeps the runtime's message
    return KFAC_ERR_CUDA;
  }
  launch_pdl(norm_backward_kernel<T, N, TPR, V, R, kDh>, dim3((unsigned)a.parts), dim3(Ring::BLOCK), smem,
             st, a);
  return KFAC_OK;
}
template <typename T, int N, int TPR, int V, int R>
kfac_status launch_backward_rows(const NormGradArgs& a, cudaStream_t st) {
  return a.dh ? launch_backward_kernel<T, N, TPR, V, R, true>(a, st)
              : launch_backward_kernel<T, N, TPR, V, R, false>(a, st);
}

// Threads per row: as in the forward pass a warp for narrow rows and 256 with as many vectors each as
// the row needs, 512 where 256 would hold too much of it; *done false: too wide.  Measured at 4096
// rows, of the copy rate: bf16 4096 wide 0.47 (two rows a round: 0.41), 8192 0.47 (256 threads: 0.43);
// fp32 4096 0.79, 8192 0.76 (read twice by the kernels below: 0.42).
template <typename T, int N> kfac_status launch_backward(const NormGradArgs& a, cudaStream_t st, bool* done) {
  constexpr bool kWhole = N * sizeof(T) == 16;
  const int64_t vecs = cdiv(a.cols, N);
  *done = true;
  if (vecs <= 32) return launch_backward_rows<T, N, 32, 1, 2>(a, st);
  if (vecs <= 64) return launch_backward_rows<T, N, 32, 2, 2>(a, st);
  if constexpr (!kWhole) {
    if (vecs <= 256) return launch_backward_rows<T, N, 32, 8, 1>(a, st);
  } else {
    if (vecs <= 256) return launch_backward_rows<T, N, 256, 1, 3>(a, st);
  }
  if (vecs <= 512) return launch_backward_rows<T, N, 256, 2, 1>(a, st);
  if constexpr (N == 8) {
    if (vecs <= 1024) return launch_backward_rows<T, N, 512, 2, 1>(a, st);
  } else {
    if (vecs <= 1024) return launch_backward_rows<T, N, 256, 4, 1>(a, st);
  }
  if constexpr (N == 4) {
    if (vecs <= 2048) return launch_backward_rows<T, N, 512, 4, 1>(a, st);
  }
  if constexpr (!kWhole) {
    if (vecs <= 2048) return launch_backward_rows<T, N, 256, 8, 1>(a, st);
    if (N == 1 && vecs <= 8192) return launch_backward_rows<T, 1, 1024, 8, 1>(a, st);
  }
  *done = false;
  return KFAC_OK;
}

// Whether rows of p are whole aligned vectors.
bool wide_ok(const void* p, int64_t ld, int64_t rows, int vec_bytes, size_t es) {
  return !p || ((uintptr_t)p % vec_bytes == 0 && (rows == 1 || ld * (int64_t)es % vec_bytes == 0));
}

}  // namespace
}  // namespace kfac

using namespace kfac;

extern "C" kfac_status kfac_rms_norm(const kfac_norm_desc* d, const void* x, const void* residual,
                                     const float* gain, void* h, void* y, float* rstd, void* q,
                                     float* scales, cudaStream_t stream) {
  if (!d || (d->dtype != KFAC_F32 && d->dtype != KFAC_BF16)) return KFAC_ERR_INVALID_ARG;
  if (d->rows < 0 || d->cols < 0 || !(d->eps >= 0.0) || !std::isfinite((float)d->eps) ||
      (d->eps > 0.0 && (float)d->eps == 0.f))
    return KFAC_ERR_INVALID_ARG;
  if (d->group != 0 && d->group != 32 && d->group != 64 && d->group != 128)
    return KFAC_ERR_INVALID_ARG;
  if (d->rows == 0 || d->cols == 0) return KFAC_OK;
  if (d->rows >= (int64_t(1) << 31) || d->cols > kMaxCols ||
      (q && d->group && cdiv(d->cols, d->group) > kMaxGroups))
    return KFAC_ERR_UNSUPPORTED;
  const size_t es = d->dtype == KFAC_BF16 ? 2 : 4;
  auto bad = [&](const void* p, int64_t ld, size_t e) {
    return p && ((uintptr_t)p % e || ld < 0 || ld > (int64_t(1) << 40) || (d->rows > 1 && ld < d->cols));
  };
  if (!x || (!y && !q) || (q && !scales) || bad(x, d->ldx, es) || bad(residual, d->ldr, es) ||
      bad(h, d->ldh, es) || bad(y, d->ldy, es) || bad(q, d->ldq, 1) || (uintptr_t)gain % 4 ||
      (uintptr_t)rstd % 4 || (uintptr_t)scales % 4)
    return KFAC_ERR_INVALID_ARG;
  if ((h == x && d->rows > 1 && d->ldh != d->ldx) ||
      (h && h == residual && d->rows > 1 && d->ldh != d->ldr) || y == x || (residual && y == residual) || (y && y == h))
    return KFAC_ERR_INVALID_ARG;
  NormArgs a{};
  a.x = x;
  a.r = residual;
  a.gain = gain;
  a.h = h;
  a.y = y;
  a.rstd = rstd;
  a.q = static_cast<uint8_t*>(q);
  a.scales = scales;
  a.rows = d->rows;
  a.ldx = d->ldx;
  a.ldr = d->ldr;
  a.ldh = d->ldh;
  a.ldy = d->ldy;
  a.ldq = d->ldq;
  a.cols = (int)d->cols;
  a.group = d->group;
  a.groups = d->group ? (int)cdiv(d->cols, d->group) : 1;
  a.shift = d->group == 32 ? 5 : d->group == 64 ? 6 : d->group == 128 ? 7 : 31;
  a.inv_cols = (float)(1.0 / (double)d->cols);
  a.eps = (float)d->eps;
  auto whole = [&](int n) {   // rows of whole vectors of n elements
    const int bytes = n * (int)es;
    return d->cols % n == 0 && wide_ok(x, d->ldx, d->rows, bytes, es) &&
           wide_ok(residual, d->ldr, d->rows, bytes, es) && wide_ok(h, d->ldh, d->rows, bytes, es) &&
           wide_ok(y, d->ldy, d->rows, bytes, es) && wide_ok(q, d->ldq, d->rows, n, 1) &&
           (uintptr_t)gain % std::min(4 * n, 16) == 0;
  };
  const bool vec = whole(16 / (int)es);
  bool done;
  if (d->dtype == KFAC_BF16)
    done = vec        ? launch_norm<__nv_bfloat16, 8>(a, stream)
           : whole(2) ? launch_norm<__nv_bfloat16, 2>(a, stream)
                      : launch_norm<__nv_bfloat16, 1>(a, stream);
  else
    done = vec        ? launch_norm<float, 4>(a, stream)
           : whole(2) ? launch_norm<float, 2>(a, stream)
                      : launch_norm<float, 1>(a, stream);
  if (!done) {
    const size_t smem = q ? (size_t)a.groups * sizeof(int) : 0;
    const dim3 grid((unsigned)a.rows), block(1024);
    if (d->dtype == KFAC_BF16) launch_pdl(norm_wide_kernel<__nv_bfloat16>, grid, block, smem, stream, a);
    else launch_pdl(norm_wide_kernel<float>, grid, block, smem, stream, a);
  }
  count_launch();
  return check_launch();
}

extern "C" kfac_status kfac_rms_norm_workspace_size(int64_t rows, int64_t cols, size_t* bytes) {
  if (!bytes || rows < 0 || cols < 0) return KFAC_ERR_INVALID_ARG;
  if (rows >= (int64_t(1) << 31) || cols > kMaxCols) return KFAC_ERR_UNSUPPORTED;
  *bytes = align_up((size_t)(backward_parts(rows, false) * 2 * cols) * sizeof(float)) +
           align_up((size_t)rows * sizeof(float));
  return KFAC_OK;
}

extern "C" kfac_status kfac_rms_norm_backward(const kfac_norm_grad_desc* d, const void* dy,
                                              const void* h, const float* gain, const float* rstd,
                                              const void* dh, void* dx, float* dgain,
                                              float* dgain_square, void* workspace,
                                              size_t workspace_bytes, cudaStream_t stream) {
  if (!d || (d->dtype != KFAC_F32 && d->dtype != KFAC_BF16)) return KFAC_ERR_INVALID_ARG;
  if (d->rows < 0 || d->cols < 0) return KFAC_ERR_INVALID_ARG;
  if ((uintptr_t)dgain % 4 || (uintptr_t)dgain_square % 4) return KFAC_ERR_INVALID_ARG;
  if (d->cols == 0 || (d->rows == 0 && !dgain && !dgain_square)) return KFAC_OK;
  if (d->rows >= (int64_t(1) << 31) || d->cols > kMaxCols) return KFAC_ERR_UNSUPPORTED;
  const size_t es = d->dtype == KFAC_BF16 ? 2 : 4;
  auto bad = [&](const void* p, int64_t ld) {
    return (uintptr_t)p % es || ld < 0 || ld > (int64_t(1) << 40) || (d->rows > 1 && ld < d->cols);
  };
  if (d->rows > 0) {
    if (!dy || !h || !rstd || bad(dy, d->lddy) || bad(h, d->ldh) || (dh && bad(dh, d->lddh)) ||
        (dx && bad(dx, d->lddx)) || (uintptr_t)gain % 4 || (uintptr_t)rstd % 4)
      return KFAC_ERR_INVALID_ARG;
    if (dx && ((dx == dy && d->rows > 1 && d->lddx != d->lddy) ||
               (dx == dh && d->rows > 1 && d->lddx != d->lddh) || dx == h))
      return KFAC_ERR_INVALID_ARG;
  }
  size_t need = 0;
  if (kfac_status e = kfac_rms_norm_workspace_size(d->rows, d->cols, &need)) return e;
  if (!workspace || (uintptr_t)workspace % kAlign || workspace_bytes < need) return KFAC_ERR_WORKSPACE;
  if (!dx && !dgain && !dgain_square) return KFAC_OK;
  NormGradArgs a{};
  a.dy = dy;
  a.h = h;
  a.dh = dh;
  a.gain = gain;
  a.rstd = rstd;
  a.dx = dx;
  a.dgain = dgain;
  a.dgain_sq = dgain_square;
  a.rows = d->rows;
  a.lddy = d->lddy;
  a.ldh = d->ldh;
  a.lddh = d->lddh;
  a.lddx = d->lddx;
  a.cols = (int)d->cols;
  a.inv_cols = (float)(1.0 / (double)d->cols);
  a.inv_rows = d->rows > 0 ? (float)(1.0 / (double)d->rows) : 0.f;
  if (dgain || dgain_square) a.part = static_cast<float*>(workspace);
  auto whole = [&](int n) {   // rows of whole vectors of n elements
    const int bytes = n * (int)es;
    return d->cols % n == 0 && wide_ok(dy, d->lddy, d->rows, bytes, es) &&
           wide_ok(h, d->ldh, d->rows, bytes, es) && wide_ok(dh, d->lddh, d->rows, bytes, es) &&
           wide_ok(dx, d->lddx, d->rows, bytes, es) && (uintptr_t)gain % std::min(4 * n, 16) == 0;
  };
  // (bf16 in pairs, 16384 x 2046: 68 us, in single elements 110; but 4096 x 8190 132 and 121, and fp32
  // 16384 x 2046 119 and 115, x 130 23 and 16)
  const bool vec = whole(16 / (int)es), pairs = es == 2 && d->cols <= 4096 && whole(2);
  a.parts = (int)backward_parts(d->rows, vec);
  int launches = 1;
  bool done;
  const kfac_status e =
      d->dtype == KFAC_BF16
          ? (vec     ? launch_backward<__nv_bfloat16, 8>(a, stream, &done)
             : pairs ? launch_backward<__nv_bfloat16, 2>(a, stream, &done)
                     : launch_backward<__nv_bfloat16, 1>(a, stream, &done))
          : (vec ? launch_backward<float, 4>(a, stream, &done) : launch_backward<float, 1>(a, stream, &done));
  if (e) return e;
  if (!done) {
    float* means = reinterpret_cast<float*>(
        static_cast<char*>(workspace) + align_up((size_t)(a.parts * 2 * d->cols) * sizeof(float)));
    const dim3 grid((unsigned)cdiv(d->cols, 256), (unsigned)a.parts);
    if (d->dtype == KFAC_BF16) {
      if (d->rows > 0)
        launch_pdl(norm_wide_dot_kernel<__nv_bfloat16>, dim3((unsigned)d->rows), dim3(1024), 0, stream, a, means);
      launch_pdl(norm_wide_backward_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, a,
                 (const float*)means);
    } else {
      if (d->rows > 0)
        launch_pdl(norm_wide_dot_kernel<float>, dim3((unsigned)d->rows), dim3(1024), 0, stream, a, means);
      launch_pdl(norm_wide_backward_kernel<float>, grid, dim3(256), 0, stream, a, (const float*)means);
    }
    launches = d->rows > 0 ? 2 : 1;
  }
  if (a.part) {
    launch_pdl(norm_parts_kernel, dim3((unsigned)cdiv(2 * (int64_t)a.cols, 32)), dim3(1024), 0, stream, a);
    ++launches;
  }
  count_launch(launches);
  return check_launch();
}
