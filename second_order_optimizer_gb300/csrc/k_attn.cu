// Cross attention: argument checks, the choice of kernels, and the kernels beside the
// products: the smallest calls that the token kernel cannot take, the joins of parts of the
// key axis, delta.
//
//   S = scale q k^T,  P = softmax over the permitted keys,  out = P v
//   dV = P^T dO,  dS = P (dO v^T - delta),  dQ = scale dS k,  dK = scale dS^T q,
//   delta = sum_d dO out.
// One pass over the keys with a running maximum m and sum l per row: a tile's
// probabilities are exp(S - m), and what was summed so far is rescaled by
// exp(m_old - m) when the maximum grows.
//
// Except in the tcgen05 kernels, query heads that share a key head are packed into one
// row axis (heads of the group x queries), so a tile of keys is loaded once for all of
// them.  Keys that are not permitted enter shared memory as zeros (or are made zeros
// there) and their scores as -infinity: what stands there in memory never meets a
// product.
#include "attn.cuh"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace kfac {
namespace attn {
namespace {

// The forward kernel for few rows and few keys that the token kernel cannot take (fp32, or
// rows that are not whole 16 bytes), on the FMA pipe: a block of 16 x 16 threads owns 16
// query rows and streams tiles of 64 keys past them; thread (ty, tx) holds row ty, keys tx +
// 16 j of a score tile and channels 4 tx + 64 c of the result.  Bound by the start of a
// block and its first tile: it has fewer steps before the first product than the kernel on
// the tensor cores, and fewer FMAs in flight for the rest (see few_rows).
template <int DP_> struct Few {
  static constexpr int BO = 16, RT = 1, BS = 64, DP = DP_;
  static constexpr int THREADS = BO / RT * 16;
  static constexpr int DPP = DP + 4;   // row pitch: float4 reads of 8 rows hit 32 banks
  static constexpr int PP = BS + 4;    // pitch of a probability row
  static constexpr int CV = DP / 64;   // float4 of channels per thread
  static constexpr int CT = BS / 16;   // keys per thread
  static constexpr size_t SMEM = sizeof(float) * (BO * DPP + 2 * BS * DPP + BO * PP) + 4 * BS;
};

// n rows x dim of global memory -> shared [n][DP + 4] fp32, zeros past dim and where
// `off` gives none (negative).  16 threads per row, four channels at a time: one
// offset per row and thread, and 16-byte loads where the rows allow (vec).
template <typename T, typename C, int N, typename Off>
__device__ __forceinline__ void load_tile(float* dst, const T* src, int dim, bool vec, Off off) {
  const int c0 = threadIdx.x % 16;
#pragma unroll 4
  for (int r = threadIdx.x / 16; r < N; r += C::THREADS / 16) {
    const int64_t o = off(r);
    const T* p = src + o;
#pragma unroll
    for (int c = c0; c < C::DP / 4; c += 16) {
      const int d = 4 * c;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (o >= 0 && d < dim) {
        if (sizeof(T) == 4 && vec) {
          v = *reinterpret_cast<const float4*>(p + d);
        } else {
          v.x = to_f32<T>(p[d]);
          if (d + 1 < dim) v.y = to_f32<T>(p[d + 1]);
          if (d + 2 < dim) v.z = to_f32<T>(p[d + 2]);
          if (d + 3 < dim) v.w = to_f32<T>(p[d + 3]);
        }
      }
      *reinterpret_cast<float4*>(dst + r * C::DPP + d) = v;
    }
  }
}
// N keys from key0 of k and v, zeros where a key is not permitted; oks[r] says
// whether it is.
template <typename T, typename C, int N>
__device__ __forceinline__ void load_keys(const Args& a, float* Ks, float* Vs, int* oks, int b, int hk,
                                          int len, int key0) {
  const int64_t kb = b * a.ks[0] + hk * a.ks[2], vb = b * a.vs[0] + hk * a.vs[2];
  load_tile<T, C, N>(Ks, static_cast<const T*>(a.k), a.dim, a.vec, [&](int r) -> int64_t {
    const bool ok = key_ok(a, b, len, key0 + r);
    if (threadIdx.x % 16 == 0) oks[r] = ok;
    return ok ? kb + (int64_t)(key0 + r) * a.ks[1] : -1;
  });
  load_tile<T, C, N>(Vs, static_cast<const T*>(a.v), a.dim, a.vec, [&](int r) -> int64_t {
    return key_ok(a, b, len, key0 + r) ? vb + (int64_t)(key0 + r) * a.vs[1] : -1;
  });
}

__device__ __forceinline__ float half_max(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// acc[i][j] = sum_d x[ty RT + i][d] y[tx + 16 j][d]
template <typename C>
__device__ __forceinline__ void dots(const float* x, const float* y, int ty, int tx,
                                     float (&acc)[C::RT][C::CT]) {
  constexpr int RT = C::RT, CT = C::CT, DPP = C::DPP;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[i][j] = 0.f;
#pragma unroll 4
  for (int d = 0; d < C::DP; d += 4) {
    float4 xr[RT], yr[CT];
#pragma unroll
    for (int i = 0; i < RT; ++i) xr[i] = *reinterpret_cast<const float4*>(x + (ty * RT + i) * DPP + d);
#pragma unroll
    for (int j = 0; j < CT; ++j) yr[j] = *reinterpret_cast<const float4*>(y + (tx + 16 * j) * DPP + d);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < CT; ++j) {
        acc[i][j] = fmaf(xr[i].x, yr[j].x, acc[i][j]);
        acc[i][j] = fmaf(xr[i].y, yr[j].y, acc[i][j]);
        acc[i][j] = fmaf(xr[i].z, yr[j].z, acc[i][j]);
        acc[i][j] = fmaf(xr[i].w, yr[j].w, acc[i][j]);
      }
  }
}

// o[i][c] += sum_k p[ty RT + i][k] y[k][4 tx + 64 c ..]
template <typename C>
__device__ __forceinline__ void add_rows(const float* p, const float* y, int ty, int tx,
                                         float4 (&o)[C::RT][C::CV]) {
  constexpr int RT = C::RT;
#pragma unroll 4
  for (int k = 0; k < C::BS; k += 4) {
    float4 pr[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) pr[i] = *reinterpret_cast<const float4*>(p + (ty * RT + i) * C::PP + k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int c = 0; c < C::CV; ++c) {
        const float4 yv = *reinterpret_cast<const float4*>(y + (k + kk) * C::DPP + 4 * tx + 64 * c);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const float w = kk == 0 ? pr[i].x : kk == 1 ? pr[i].y : kk == 2 ? pr[i].z : pr[i].w;
          o[i][c].x = fmaf(w, yv.x, o[i][c].x);
          o[i][c].y = fmaf(w, yv.y, o[i][c].y);
          o[i][c].z = fmaf(w, yv.z, o[i][c].z);
          o[i][c].w = fmaf(w, yv.w, o[i][c].w);
        }
      }
  }
}
template <typename C>
__device__ __forceinline__ void clear(float4 (&o)[C::RT][C::CV]) {
#pragma unroll
  for (int i = 0; i < C::RT; ++i)
#pragma unroll
    for (int c = 0; c < C::CV; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
}

template <typename T>
__device__ __forceinline__ void store4(T* dst, int d, int dim, float4 v, float f) {
  if (d < dim) dst[d] = (T)(v.x * f);
  if (d + 1 < dim) dst[d + 1] = (T)(v.y * f);
  if (d + 2 < dim) dst[d + 2] = (T)(v.z * f);
  if (d + 3 < dim) dst[d + 3] = (T)(v.w * f);
}

// grid: (row tiles x splits, kv_heads, batch)
template <typename T, typename C>
__global__ void __launch_bounds__(C::THREADS) few_rows_kernel(const __grid_constant__ Args a) {
  constexpr int RT = C::RT, CV = C::CV, CT = C::CT, BO = C::BO, BS = C::BS;
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Ks = Qs + BO * C::DPP;
  float* Vs = Ks + BS * C::DPP;
  float* Ps = Vs + BS * C::DPP;
  int* oks = reinterpret_cast<int*>(Ps + BO * C::PP);
  pdl_wait();
  pdl_trigger();
  const int tile = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  const int hk = blockIdx.y, b = blockIdx.z, r0 = tile * BO;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int len = walk_end(a, b);
  const int tiles = (len + BS - 1) / BS;
  const int t0 = (int)((int64_t)tiles * split / a.splits);
  const int t1 = (int)((int64_t)tiles * (split + 1) / a.splits);
  load_tile<T, C, BO>(Qs, static_cast<const T*>(a.q), a.dim, a.vec, [&](int r) -> int64_t {
    return r0 + r < a.rows ? row_offset(a, a.qs, b, hk, r0 + r) : -1;
  });
  float m[RT], l[RT];
  float4 o[RT][CV];
  clear<C>(o);
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
  const float c2 = a.scale * kLog2e;
  for (int t = t0; t < t1; ++t) {
    __syncthreads();
    load_keys<T, C, BS>(a, Ks, Vs, oks, b, hk, len, t * BS);
    __syncthreads();
    float s[RT][CT];
    dots<C>(Qs, Ks, ty, tx, s);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < CT; ++j) {
        s[i][j] = oks[tx + 16 * j] ? s[i][j] * c2 : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
      const float mn = fmaxf(m[i], half_max(top));
      const float base = mn == -INFINITY ? 0.f : mn;   // nothing permitted so far
      const float f = exp2f(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < CT; ++j) {
        const float p = exp2f(s[i][j] - base);
        sum += p;
        Ps[(ty * RT + i) * C::PP + tx + 16 * j] = p;
      }
      l[i] = l[i] * f + half_sum(sum);
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < CV; ++c) {
        o[i][c].x *= f;
        o[i][c].y *= f;
        o[i][c].z *= f;
        o[i][c].w *= f;
      }
    }
    __syncwarp();   // a row's probabilities come from its own half warp
    add_rows<C>(Ps, Vs, ty, tx, o);
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = r0 + ty * RT + i;
    if (r >= a.rows) continue;
    const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);
    const float lse = l[i] == 0.f ? -INFINITY : m[i] * kLn2 + logf(l[i]);
    if (a.splits == 1) {
      T* dst = static_cast<T*>(a.out) + row_offset(a, a.os, b, hk, r);
#pragma unroll
      for (int c = 0; c < CV; ++c) store4(dst, 4 * tx + 64 * c, a.dim, o[i][c], inv);
      if (a.lse && tx == 0) a.lse[((int64_t)b * a.kv_heads + hk) * a.rows + r] = lse;
    } else {
      const int64_t at = (((int64_t)split * a.batch + b) * a.kv_heads + hk) * a.rows + r;
#pragma unroll
      for (int c = 0; c < CV; ++c) store4(a.part_o + at * a.dim, 4 * tx + 64 * c, a.dim, o[i][c], inv);
      if (tx == 0) a.part_lse[at] = lse;
    }
  }
}

// Joins the parts of the key axis: out = sum_s w_s o_s, w_s = exp(lse_s - lse).  One block
// of four warps per row, a quarter of the parts each (the sums of a quarter in order, then
// the quarters in order).  [batch][kv_heads][rows] is [batch][heads][len_q], lse's layout.
template <typename T>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ Args a) {
  __shared__ float acc_s[4][128], total_s[4];
  pdl_wait();
  pdl_trigger();
  const int64_t n = (int64_t)a.batch * a.kv_heads * a.rows;
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  float top = -INFINITY;
  for (int s = lane; s < a.splits; s += 32) top = fmaxf(top, a.part_lse[s * n + row]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float base = top == -INFINITY ? 0.f : top;
  float total = 0.f;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = warp; s < a.splits; s += 4) {
    const float w = exp2f((a.part_lse[s * n + row] - base) * kLog2e);
    total += w;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int d = lane + 32 * c;
      if (d < a.dim) acc[c] = fmaf(w, a.part_o[(s * n + row) * a.dim + d], acc[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) acc_s[warp][lane + 32 * c] = acc[c];
  if (lane == 0) total_s[warp] = total;
  __syncthreads();
  total = (total_s[0] + total_s[1]) + (total_s[2] + total_s[3]);
  const float inv = total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);
  const int r = (int)(row % a.rows), hk = (int)(row / a.rows % a.kv_heads);
  const int b = (int)(row / a.rows / a.kv_heads), d = threadIdx.x;
  if (d < a.dim)
    static_cast<T*>(a.out)[row_offset(a, a.os, b, hk, r) + d] =
        (T)(((acc_s[0][d] + acc_s[1][d]) + (acc_s[2][d] + acc_s[3][d])) * inv);
  if (a.lse && d == 0) a.lse[row] = total == 0.f ? -INFINITY : base + logf(total);
}

// delta[b][h][i] = sum_d dout out, in fp32.  L lanes per row (L divides 32), each taking
// pieces of 16 bytes (vec) or one channel at a time.
template <typename T, int L>
__global__ void __launch_bounds__(256) delta_kernel(const __grid_constant__ Args a) {
  pdl_wait();
  pdl_trigger();
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t n = (int64_t)a.batch * a.heads * a.len_q;
  const int64_t row = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  const int lane = threadIdx.x % L;
  float s = 0.f;
  if (row < n) {
    const int i = (int)(row % a.len_q);
    const int64_t bh = row / a.len_q;
    const int h = (int)(bh % a.heads), b = (int)(bh / a.heads);
    const T* o = static_cast<const T*>(a.o) + b * a.os[0] + i * a.os[1] + h * a.os[2];
    const T* g = static_cast<const T*>(a.dout) + b * a.dos[0] + i * a.dos[1] + h * a.dos[2];
    if (a.vec) {
      struct alignas(16) P { T v[V]; };
      for (int d = V * lane; d < a.dim; d += V * L) {
        const P x = *reinterpret_cast<const P*>(o + d), y = *reinterpret_cast<const P*>(g + d);
#pragma unroll
        for (int e = 0; e < V; ++e) s = fmaf(to_f32<T>(x.v[e]), to_f32<T>(y.v[e]), s);
      }
    } else {
      for (int d = lane; d < a.dim; d += L) s = fmaf(to_f32<T>(o[d]), to_f32<T>(g[d]), s);
    }
  }
#pragma unroll
  for (int k = L / 2; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
  if (lane == 0 && row < n) a.delta[row] = s;
}

// Sums the parts of the gradients that have several, in their order.  One warp per row:
// dQ's rows first (when it has parts), then dK's and dV's.
template <typename T>
__global__ void __launch_bounds__(256) sum_parts_kernel(const __grid_constant__ Args a) {
  pdl_wait();
  pdl_trigger();
  const int64_t nq = a.dq_splits > 1 ? (int64_t)a.batch * a.kv_heads * a.rows : 0;
  const int64_t nk = a.dkv_splits > 1 ? (int64_t)a.batch * a.kv_heads * a.len_kv : 0;
  int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (row >= nq + 2 * nk) return;
  const float* src;
  T* dst;
  int64_t n;
  int splits;
  float f = a.scale;
  if (row < nq) {
    src = a.part_dq;
    n = nq;
    splits = a.dq_splits;
    const int r = (int)(row % a.rows);
    const int64_t bh = row / a.rows;
    dst = static_cast<T*>(a.dq) + row_offset(a, a.dqs, (int)(bh / a.kv_heads), (int)(bh % a.kv_heads), r);
  } else {
    row -= nq;
    const bool v = row >= nk;
    if (v) row -= nk, f = 1.f;
    src = v ? a.part_dv : a.part_dk;
    n = nk;
    splits = a.dkv_splits;
    const int64_t key = row % a.len_kv, bh = row / a.len_kv;
    const int64_t(&st)[3] = v ? a.dvs : a.dks;
    dst = static_cast<T*>(v ? a.dv : a.dk) + bh / a.kv_heads * st[0] + key * st[1] + bh % a.kv_heads * st[2];
  }
  for (int d = lane; d < a.dim; d += 32) {
    float s = 0.f;
    for (int i = 0; i < splits; ++i) s += src[(i * n + row) * a.dim + d];
    dst[d] = (T)(s * f);
  }
}

template <typename T, typename C>
kfac_status launch_few_rows(const Args& a, cudaStream_t st) {
  static OncePerDevice once;
  const kfac_status e = allow_smem(once, few_rows_kernel<T, C>, C::SMEM);
  if (e != KFAC_OK) return e;
  const dim3 grid((unsigned)(cdiv(a.rows, C::BO) * a.splits), a.kv_heads, a.batch);
  launch_pdl(few_rows_kernel<T, C>, grid, dim3(C::THREADS), C::SMEM, st, a);
  count_launch();
  return check_launch();
}

template <typename T>
kfac_status launch_combine(const Args& a, cudaStream_t st) {
  const int64_t n = (int64_t)a.batch * a.kv_heads * a.rows;
  launch_pdl(combine_kernel<T>, dim3((unsigned)n), dim3(128), 0, st, a);
  count_launch();
  return check_launch();
}

// Rows that start at multiples of 16 bytes (v elements) and hold whole ones.
bool vec_rows(const void* p, const int64_t* s, int rows, int heads, int batch, int dim, int v) {
  return dim % v == 0 && (uintptr_t)p % 16 == 0 && (batch <= 1 || s[0] % v == 0) &&
         (rows <= 1 || s[1] % v == 0) && (heads <= 1 || s[2] % v == 0);
}

// Up to 16 rows against up to kFewKeys keys of all batch entries and key heads: there a call
// is one wave of blocks of a tile or two.  One row, batch entries x key heads x keys, fp32,
// us of few_rows_kernel and of f32_forward_kernel:
//   64 channels   16 x 64: 6.6, 7.9; 16 x 256: 8.7, 10.3; 4 x 1024: 9.5, 10.9; 16 x 333: 9.1,
//                 10.6; 16 x 512: 11.7, 10.8; 4 x 2048: 12.7, 11.7; 256 x 256: 32, 18
//   128 channels  16 x 64: 9.1, 11.2; 16 x 256: 14.2, 14.0; 4 x 1024: 14.9, 14.5;
//                 64 x 128: 15.3, 14.6; 256 x 256: 61, 37; 128 x 8192: 924, 537
constexpr int64_t kFewKeys = 6144;
bool few_rows(int64_t rows, int64_t batch, int64_t kv_heads, int64_t len_kv) {
  return rows <= 16 && batch * kv_heads * len_kv <= kFewKeys;
}

template <typename T>
kfac_status plain_forward(Args a, cudaStream_t st) {
  a.vec = vec_rows(a.q, a.qs, a.len_q, a.heads, a.batch, a.dim, 4) &&
          vec_rows(a.k, a.ks, a.len_kv, a.kv_heads, a.batch, a.dim, 4) &&
          vec_rows(a.v, a.vs, a.len_kv, a.kv_heads, a.batch, a.dim, 4);
  kfac_status e;
  if (few_rows(a.rows, a.batch, a.kv_heads, a.len_kv))
    e = a.dim <= 64 ? launch_few_rows<T, Few<64>>(a, st)
                    : launch_few_rows<T, Few<128>>(a, st);
  else
    e = f32_forward<T>(a, st);
  if (e == KFAC_OK && a.splits > 1) e = launch_combine<T>(a, st);
  return e;
}

template <typename T>
kfac_status launch_delta(Args a, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t n = (int64_t)a.batch * a.heads * a.len_q;
  a.vec = vec_rows(a.o, a.os, a.len_q, a.heads, a.batch, a.dim, V) &&
          vec_rows(a.dout, a.dos, a.len_q, a.heads, a.batch, a.dim, V);
  launch_pdl(delta_kernel<T, 8>, dim3((unsigned)cdiv(n, 32)), dim3(256), 0, st, a);
  count_launch();
  return check_launch();
}

template <typename T>
kfac_status backward(Args a, cudaStream_t st) {
  const int64_t n = (int64_t)a.batch * a.heads * a.len_q;
  const bool bf16 = sizeof(T) == 2, tc = bf16 && tc_backward_ok(a);
  a.vec = vec_rows(a.q, a.qs, a.len_q, a.heads, a.batch, a.dim, 4) &&
          vec_rows(a.dout, a.dos, a.len_q, a.heads, a.batch, a.dim, 4) &&
          vec_rows(a.k, a.ks, a.len_kv, a.kv_heads, a.batch, a.dim, 4) &&
          vec_rows(a.v, a.vs, a.len_kv, a.kv_heads, a.batch, a.dim, 4);
  if (n > 0) {
    // bf16: out is rounded, and with few keys delta has to be better than that
    kfac_status e = KFAC_OK;
    const bool all_few = bf16 && a.len_kv <= kExactKeys;
    if (!all_few) e = launch_delta<T>(a, st);
    if (e == KFAC_OK && bf16 && (all_few || a.kv_len || a.key_mask)) e = tc ? delta_keys(a, st) : f32_delta(a, st);
    if (e != KFAC_OK) return e;
  }
  kfac_status e;
  if (tc) {
    e = tc_backward(a, st);
  } else {
    e = f32_backward<T>(a, st);
  }
  const int64_t sums = (a.dq_splits > 1 ? n : 0) +
                       (a.dkv_splits > 1 ? 2 * (int64_t)a.batch * a.kv_heads * a.len_kv : 0);
  if (e != KFAC_OK || sums == 0) return e;
  launch_pdl(sum_parts_kernel<T>, dim3((unsigned)cdiv(sums, 8)), dim3(256), 0, st, a);
  count_launch();
  return check_launch();
}

// Parts of the key axis for `ctas` blocks of the unsplit product: enough for `per_sm`
// blocks per SM, no part shorter than a tile of `tile` keys.
int pick_splits(int64_t ctas, int per_sm, int len_kv, int tile) {
  const int64_t want = per_sm * num_sms() / std::max<int64_t>(ctas, 1);
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, cdiv(len_kv, tile), 64}));
}

int plain_splits(const kfac_attention_desc& d) {
  const int rows = d.heads / d.kv_heads * d.len_q;
  const bool few = few_rows(rows, d.batch, d.kv_heads, d.len_kv);   // (no more tiles than blocks fit)
  // as many blocks as are resident
  const int per_sm = d.head_dim <= 64 ? 4 : 2;
  return pick_splits((int64_t)cdiv(rows, few ? 16 : 64) * d.kv_heads * d.batch, per_sm, d.len_kv, 64);
}
// Rows (keys, or queries of a group) that one tensor-core accumulator sums.  Its additions
// round towards zero, about half an ulp each: of a sum of like signs that takes away 4e-5
// after 8192 rows, 2.2e-4 after 32768, and 3.3e-3, more than the result's rounding to bf16,
// after 524288 (measured: out, dV, single tokens).  Longer walks come in parts, which are
// summed in fp32 registers: 16 heads x 128, 8192 queries, 65536 keys: forward 2.65 ms in one
// part and in two, backward 8.3 and 8.4 ms; 4 heads that share a key head x 131072 queries,
// 2048 keys, 64 channels: backward 1.71 and 1.74 ms.
constexpr int kWalkRows = 32768;
// (a part of fewer than 512 keys costs more to join than it saves: 2 x 300 queries, 300
// keys, 8 heads x 64: 10 us unsplit, 15 us in three parts)
int tc_splits(const kfac_attention_desc& d) {
  const int tiles = tc_forward_tiles(d.head_dim, d.len_q, d.len_kv);
  const int fill = pick_splits((int64_t)cdiv(d.len_q, 128 * tiles) * d.heads * d.batch,
                               tiles == 1 ? 2 : 1, d.len_kv, 512);
  return std::max(fill, (int)cdiv(d.len_kv, kWalkRows));
}
// The form of the forward pass for bf16 rows that TMA and 16-byte loads can address.  The
// token kernel passes k and v by once per 16 packed rows of a key head, the tcgen05 kernel once
// per query head (in tiles of 128 or 256 queries): the first while it has at most 3/4 as many
// passes, or one.  Batch entries x queries x keys (r: ragged), heads on key heads x channels, us
// of the token and of the tcgen05 kernel:
//   1 head per key head  16 x 4 x 1024, 8 x 64: 11.0, 14.5; 8 x 16 x 4096 r, 8 x 128: 25.6, 23.9;
//                        8 x 8 x 4096, 8 x 128: 40.7, 28.9; 16 x 32 x 1024, 8 x 64: 22.0, 18.3;
//                        64 x 32 x 512, 8 x 64: 33, 20; 8 x 64 x 4096, 8 x 128: 117, 35
//   4                    16 x 4 x 4096, 16 x 128: 44, 54; 16 x 8: 47, 54; 16 x 12: 65, 54;
//                        32 x 12 x 512 r, 16 x 64: 13.4, 15.8; 16 x 16 x 4096: 117, 54
//   8                    16 x 4 x 4096, 32 x 128: 47, 104; 16 x 12: 118, 104, r 68, 80;
//                        16 x 16: 171, 104, r 89, 71
//   16                   16 x 8 x 4096, 16 x 128: 47, 53; 64 x 12 x 1024 r, 16 x 64: 27, 37;
//                        16 x 16 x 4096: 116, 53
// (A single query on one head per key head is near even, 0.7 to 1.4 times; it stays with the
// token kernel, which needs no tensor maps, 1 us of the host's time.)
bool token_sizes(const kfac_attention_desc& d) {
  const int64_t group = d.heads / d.kv_heads;
  return d.dtype == KFAC_BF16 && cdiv(group * d.len_q, 16) <= std::max<int64_t>(1, 3 * group / 4);
}
// Parts of the key axis for the token kernel: as many blocks as are resident at once, and no
// more for equal lengths, where a second wave of a few blocks costs as much as a whole one
// (32 x 8192 keys on 4 key heads x 128: 84 us in 3 parts and 113 us in 4).  Ragged lengths
// leave blocks idle, which the blocks of a second wave fill, if the walks are longer than a
// wave's cost of about 5 us (128 channels, walks x keys: parts and us; the waves' choice
// first): 128 x 512, 3: 11.0, 4: 13.3; 128 x 2048, 4: 20.8, 3: 24.0, 6: 25.7;
// 256 x 4096, 3: 46.3, 2: 59.5, 4: 52.5; 128 x 8192, 6: 44.2, 4: 58.0, 8: 51.2.
// Each warp has at least one step of 16 keys and at most kWalkRows keys.  Up to kTokenCluster parts are joined in a
// cluster, more are fixed lengths, which are even by themselves.
constexpr int kTokenWaves1 = 1024, kTokenWaves2 = 4096;   // keys: 1 wave below, 1.5 from
int token_splits(const kfac_attention_desc& d, bool ragged, int* part_keys) {
  const int64_t ctas = std::max<int64_t>(
      1, cdiv((int64_t)d.heads / d.kv_heads * d.len_q, 16) * d.kv_heads * d.batch);
  const int step = 16 * kTokenWarps;
  const int64_t most = std::max<int64_t>(1, cdiv(d.len_kv, step)), slots = kTokenPerSm * num_sms();
  int64_t parts = std::max<int64_t>(1, slots / ctas);
  const bool clustered = parts <= kTokenCluster;
  if (ragged && d.batch > 1 && d.len_kv >= kTokenWaves1)
    parts = cdiv(d.len_kv < kTokenWaves2 ? slots : slots + slots / 2, ctas);
  if (clustered) parts = std::min<int64_t>(parts, kTokenCluster);
  parts = std::max(parts, cdiv(d.len_kv, kTokenWarps * kWalkRows));
  parts = std::min(parts, most);
  *part_keys = d.len_kv;
  if (parts > kTokenCluster) {
    *part_keys = (int)(cdiv(cdiv(d.len_kv, parts), step) * step);
    parts = cdiv(d.len_kv, *part_keys);
  }
  return (int)parts;
}

bool valid_desc(const kfac_attention_desc* d) {
  if (!d || (d->dtype != KFAC_F32 && d->dtype != KFAC_BF16)) return false;
  if (d->batch < 0 || d->len_q < 0 || d->len_kv < 0 || d->heads < 1 || d->kv_heads < 1) return false;
  if (d->heads % d->kv_heads || d->heads > 65535 || d->kv_heads > 65535 || d->batch > 65535)
    return false;
  if (d->head_dim < 1) return false;
  if (!std::isfinite(d->scale) || d->scale < 0.f) return false;
  // packed rows, tiles and rows of the statistics are counted in 32 bits
  if ((int64_t)d->heads * std::max(d->len_q, 1) > (int64_t(1) << 30) || d->len_kv > (1 << 30))
    return false;
  if ((int64_t)d->batch * d->heads * d->len_q > (int64_t(1) << 31)) return false;
  return true;
}

size_t part_bytes(const kfac_attention_desc& d, int splits) {
  return splits > 1 ? align_up((size_t)splits * d.batch * d.heads * d.len_q * (d.head_dim + 1) *
                               sizeof(float))
                    : 0;
}

// Parts of the backward pass's loops.  A dK/dV block owns `own` keys and walks the group's
// queries in steps (four products each), a dQ block owns as many queries and walks the
// keys (three).  Where one block's walk is longer than its share of the whole work, it is
// split, into at most 32 pieces of at least four steps; the sums then take a launch more.  us with
// pieces of 2, 4 and 8 steps at least, queries x keys (channels): bf16 2500 x 40 (128): 30, 26, 25;
// 20 x 3100 (64): 13.0, 12.0, 14.7; 64 x 8192 (128): 35, 25, 23; fp32 20 x 3100 (64): 33, 36, 44;
// 2500 x 40 (128): 101, 101, 135.  With 16, 32 and 64 pieces at most: bf16 128 x 32768 (64): 32, 32,
// 44; 65536 x 64 (64): 56, 49, 60; fp32 8192 x 64 (128): 241, 153, 124; 128 x 32768 (64): 282, 184, 165.
// The tensor-core kernels' accumulators walk no further than kWalkRows.
// tc: of the tensor-core kernels (bf16), else of the fp32 ones.
void backward_splits(const kfac_attention_desc& d, Args& a, bool tc) {
  const int own = tc ? 128 : 64, step = tc ? 128 : 32, per_sm = tc ? 1 : 2;
  const int64_t group = d.heads / d.kv_heads;
  const int64_t rows = group * d.len_q, blocks_q = tc ? group * cdiv(d.len_q, own) : cdiv(rows, own);
  const int64_t steps_q = tc ? blocks_q : cdiv(rows, step), steps_k = cdiv(d.len_kv, step);
  const int64_t work = (4 * cdiv(d.len_kv, own) * steps_q + 3 * blocks_q * steps_k) * d.kv_heads * d.batch;
  const int64_t share = std::max<int64_t>(1, work / (per_sm * num_sms()));
  auto parts = [&](int64_t steps, int64_t weight) {
    const int64_t fill = std::min<int64_t>({cdiv(steps * weight, share), steps / 4, 32});
    return (int)std::max<int64_t>({1, fill, tc ? cdiv(steps, kWalkRows / step) : 1});
  };
  a.dkv_splits = parts(steps_q, 4);
  a.dq_splits = parts(steps_k, 3);
}
// Bytes of the backward pass's workspace; places its pieces at `ws`.
size_t backward_bytes(const kfac_attention_desc& d, Args& a, char* ws) {
  size_t at = 0;
  auto take = [&](size_t floats) {
    float* p = reinterpret_cast<float*>(ws + at);
    at += align_up(floats * sizeof(float));
    return p;
  };
  const size_t q = (size_t)d.batch * d.heads * d.len_q, k = (size_t)d.batch * d.kv_heads * d.len_kv;
  a.delta = take(q);
  a.part_dq = a.dq_splits > 1 ? take(a.dq_splits * q * d.head_dim) : nullptr;
  a.part_dk = a.dkv_splits > 1 ? take(a.dkv_splits * k * d.head_dim) : nullptr;
  a.part_dv = a.dkv_splits > 1 ? take(a.dkv_splits * k * d.head_dim) : nullptr;
  return at;
}

size_t workspace_bytes_for(const kfac_attention_desc& d, bool backward) {
  int splits = plain_splits(d), keys;   // whichever form the tensors' layouts allow
  if (d.dtype == KFAC_BF16)
    splits = std::max(splits, token_sizes(d) ? token_splits(d, true, &keys) : tc_splits(d));
  const size_t fwd = part_bytes(d, splits);
  if (!backward) return fwd;
  Args a{};
  backward_splits(d, a, false);
  const size_t bytes = std::max(fwd, backward_bytes(d, a, nullptr));
  if (d.dtype != KFAC_BF16) return bytes;
  backward_splits(d, a, true);
  return std::max(bytes, backward_bytes(d, a, nullptr));
}

struct Tensor {
  const void* p;
  const int64_t* s;
  int64_t rows, heads;
  bool output;
};

bool valid_tensor(const kfac_attention_desc& d, const Tensor& t) {
  const size_t es = d.dtype == KFAC_BF16 ? 2 : 4;
  const int64_t n[3] = {d.batch, t.rows, t.heads};
  if (d.batch == 0 || t.rows == 0) return true;   // nothing there to read or write
  if (!t.p || (uintptr_t)t.p % es) return false;
  for (int i = 0; i < 3; ++i) {
    if (t.s[i] < 0) return false;
    // an output's rows may not overlap; an input's axis may be broadcast
    if (t.output && n[i] > 1 && t.s[i] < d.head_dim) return false;
  }
  return true;
}

void fill(Args& a, const kfac_attention_desc& d) {
  a.batch = d.batch;
  a.len_q = d.len_q;
  a.len_kv = d.len_kv;
  a.heads = d.heads;
  a.kv_heads = d.kv_heads;
  a.group = d.heads / d.kv_heads;
  a.dim = d.head_dim;
  a.rows = a.group * d.len_q;
  a.scale = d.scale > 0.f ? d.scale : (float)(1.0 / std::sqrt((double)d.head_dim));
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = d.q_stride[i];
    a.ks[i] = d.k_stride[i];
    a.vs[i] = d.v_stride[i];
    a.os[i] = d.out_stride[i];
  }
}

}  // namespace
}  // namespace attn
}  // namespace kfac

using namespace kfac;
using namespace kfac::attn;

extern "C" {

kfac_status kfac_cross_attention_workspace_size(const kfac_attention_desc* d, int backward,
                                                size_t* bytes) {
  if (!valid_desc(d) || !bytes || (backward != 0 && backward != 1)) return KFAC_ERR_INVALID_ARG;
  if (d->head_dim > 128) return KFAC_ERR_UNSUPPORTED;
  *bytes = workspace_bytes_for(*d, backward != 0);
  return KFAC_OK;
}

kfac_status kfac_cross_attention(const kfac_attention_desc* d, const void* q, const void* k,
                                 const void* v, const int* kv_len, const uint8_t* key_mask,
                                 void* out, float* lse, void* workspace, size_t workspace_bytes,
                                 cudaStream_t stream) {
  if (!valid_desc(d)) return KFAC_ERR_INVALID_ARG;
  if (d->head_dim > 128) return KFAC_ERR_UNSUPPORTED;
  const Tensor ts[] = {{q, d->q_stride, d->len_q, d->heads, false},
                       {k, d->k_stride, d->len_kv, d->kv_heads, false},
                       {v, d->v_stride, d->len_kv, d->kv_heads, false},
                       {out, d->out_stride, d->len_q, d->heads, true}};
  for (const Tensor& t : ts)
    if (!valid_tensor(*d, t)) return KFAC_ERR_INVALID_ARG;
  if ((uintptr_t)kv_len % 4 || (uintptr_t)lse % 4) return KFAC_ERR_INVALID_ARG;
  const size_t need = workspace_bytes_for(*d, false);
  if (need && (!workspace || (uintptr_t)workspace % kAlign || workspace_bytes < need))
    return KFAC_ERR_WORKSPACE;
  if (d->batch == 0 || d->len_q == 0) return KFAC_OK;
  Args a{};
  fill(a, *d);
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.lse = lse;
  a.kv_len = kv_len;
  a.key_mask = key_mask;
  const bool tc = d->dtype == KFAC_BF16 && tc_forward_ok(a), token = tc && token_sizes(*d);
  a.splits = token ? token_splits(*d, kv_len != nullptr, &a.part_keys) : tc ? tc_splits(*d) : plain_splits(*d);
  // The order costs each block a look at all lengths, which short walks do not win back.  Tokens x
  // keys (ragged), us without and with it: 16 heads on 4 x 128: 128 x 64: 8.7, 11.2; 128 x 512:
  // 19.8, 20.2; 128 x 1024: 31.2, 33.1; 128 x 4096: 103, 93; 16 on 8 x 64: 100 x 256: 11.9, 13.3;
  // 100 x 512: 17.4, 16.5; 100 x 2048: 47.9, 39.2
  a.longest_first = token && kv_len && d->batch > 1 && d->batch <= kTokenOrdered && d->len_kv >= 512 &&
                    cdiv(a.rows, 16) * a.splits * (int64_t)d->kv_heads * d->batch > kTokenPerSm * num_sms();
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = a.part_o + (size_t)a.splits * d->batch * d->heads * d->len_q * d->head_dim;
  if (tc) {
    kfac_status e = token ? token_forward(a, stream) : tc_forward(a, stream);
    const bool joined = token && a.splits <= kTokenCluster;
    if (e == KFAC_OK && a.splits > 1 && !joined) e = launch_combine<__nv_bfloat16>(a, stream);
    return e;
  }
  return d->dtype == KFAC_BF16 ? plain_forward<__nv_bfloat16>(a, stream) : plain_forward<float>(a, stream);
}

kfac_status kfac_cross_attention_backward(const kfac_attention_desc* d,
                                          const kfac_attention_grad_desc* g, const void* dout,
                                          const void* q, const void* k, const void* v,
                                          const void* out, const float* lse, const int* kv_len,
                                          const uint8_t* key_mask, void* dq, void* dk, void* dv,
                                          void* workspace, size_t workspace_bytes,
                                          cudaStream_t stream) {
  if (!valid_desc(d) || !g) return KFAC_ERR_INVALID_ARG;
  if (d->head_dim > 128) return KFAC_ERR_UNSUPPORTED;
  const Tensor ts[] = {{q, d->q_stride, d->len_q, d->heads, false},
                       {k, d->k_stride, d->len_kv, d->kv_heads, false},
                       {v, d->v_stride, d->len_kv, d->kv_heads, false},
                       {out, d->out_stride, d->len_q, d->heads, false},
                       {dout, g->dout_stride, d->len_q, d->heads, false},
                       {dq, g->dq_stride, d->len_q, d->heads, true},
                       {dk, g->dk_stride, d->len_kv, d->kv_heads, true},
                       {dv, g->dv_stride, d->len_kv, d->kv_heads, true}};
  for (const Tensor& t : ts)
    if (!valid_tensor(*d, t)) return KFAC_ERR_INVALID_ARG;
  if ((d->batch && d->len_q && !lse) || (uintptr_t)kv_len % 4 || (uintptr_t)lse % 4)
    return KFAC_ERR_INVALID_ARG;
  const size_t need = workspace_bytes_for(*d, true);
  if (need && (!workspace || (uintptr_t)workspace % kAlign || workspace_bytes < need))
    return KFAC_ERR_WORKSPACE;
  if (d->batch == 0 || (d->len_q == 0 && d->len_kv == 0)) return KFAC_OK;
  Args a{};
  fill(a, *d);
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = out;
  a.dout = dout;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.lse_in = lse;
  a.kv_len = kv_len;
  a.key_mask = key_mask;
  for (int i = 0; i < 3; ++i) {
    a.dos[i] = g->dout_stride[i];
    a.dqs[i] = g->dq_stride[i];
    a.dks[i] = g->dk_stride[i];
    a.dvs[i] = g->dv_stride[i];
  }
  backward_splits(*d, a, d->dtype == KFAC_BF16 && tc_backward_ok(a));
  backward_bytes(*d, a, static_cast<char*>(workspace));
  return d->dtype == KFAC_BF16 ? backward<__nv_bfloat16>(a, stream) : backward<float>(a, stream);
}

}  // extern "C"
