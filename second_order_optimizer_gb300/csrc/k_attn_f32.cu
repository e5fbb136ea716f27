// Cross attention of fp32 inputs (and of bf16 rows that the tensor-memory accelerator
// cannot address): forward but for the smallest calls, and the backward pass.
//
// Products run on the tensor cores with fp32 accuracy.  Each operand v enters as its
// TF32 rounding h and the remainder r = v - h (exact in fp32); x y = h h' + (h r' + r h'),
// three mma.sync m16n8k8 products, the dropped r r' about 2^-22 of the whole.  h h' and
// the small cross terms have accumulators of their own, and no accumulator outlives a
// tile: the tensor cores' additions round towards zero, and what is summed over tiles is
// summed in fp32 registers.  (On the FMA pipe the same tiles were bound by shared-memory
// reads, 8 16-byte loads per 64 FMAs: 25 TFLOP/s.)  4 x 1024 queries and keys, 8 heads on 4 x
// 128: forward 406 us, 42 TFLOP/s; backward 1660 us; on 8 x 64: 218 and 741 us.  Bound by issue at
// 8 to 16 warps per SM: the three products alone could run at 98 TFLOP/s.
//
// bf16 values are TF32 values: their scores take one product, and P or dS with one of them
// two (h y + r y).
//
// A block owns 64 rows (queries, or keys for dK and dV), 16 per warp, and streams tiles
// of BS rows of the other side past them, two buffers of them in shared memory, the next one
// on its way (cp.async) while the present one is multiplied.  They lie there as they are and
// are split by each warp that reads them: storing both parts instead halves neither the
// issue slots nor the time, and took the room of the second buffer (8 x 64: 257 and 810 us; 8
// x 32: forward 210 us, now 130).  The scores of a warp's rows stay in its
// registers: the columns that a lane holds of S are the k slots that it supplies to the
// next product, once keys are taken in that order (slot t of eight: key 2t, slot t + 4:
// key 2t + 1).  Shared rows have a pitch of 4 mod 32 floats, for which both kinds of
// 16-byte reads are free of bank conflicts: rows of a score product (lane (g, t): row g,
// channels 8t + 4j of 32) and rows of a value product (row 2t or 2t + 1, channels 4g).
#include "attn.cuh"
#include "tc_prims.cuh"

#include <algorithm>
#include <type_traits>

namespace kfac {
namespace attn {
namespace {

constexpr int kRows = 64;        // own rows of a block
constexpr int kF32Threads = 128;
constexpr uint32_t kAll = 0xffffffffu;

template <int BS_, int DP_> struct Cfg {
  static constexpr int BS = BS_, DP = DP_, DPP = DP + 4;
  static constexpr int NT = BS / 8;    // 8-column tiles of a score row
  static constexpr int NB = DP / 32;   // 32-channel blocks
  static constexpr int TILE = BS * DPP;   // floats of a streamed tile
  static constexpr size_t FWD = sizeof(float) * (kRows * DPP + 4 * TILE) + 4 * 2 * BS;
  static constexpr size_t BWD = sizeof(float) * (2 * kRows * DPP + 4 * TILE) + 4 * (4 * BS + kRows);
};

// v = h + r: h rounded to TF32's 11 bits (half away from zero, by integer addition), r
// exact.  An infinite v has r = NaN here ...
struct Split { uint32_t h, r; };
__device__ __forceinline__ Split split(float v) {
  const uint32_t h = (__float_as_uint(v) + 0x1000u) & 0xffffe000u;
  return {h, __float_as_uint(v - __uint_as_float(h))};
}
// ... and 0 here, where the infinity would otherwise be lost: in streamed tiles.
__device__ __forceinline__ Split split_inf(float v) {
  Split s = split(v);
  if ((s.h & 0x7fffffffu) == 0x7f800000u) s.r = 0u;
  return s;
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma3(float (&hi)[4], float (&lo)[4], const Split (&a)[4], Split b0,
                                     Split b1) {
  mma_tf32(lo, a[0].r, a[1].r, a[2].r, a[3].r, b0.h, b1.h);
  mma_tf32(lo, a[0].h, a[1].h, a[2].h, a[3].h, b0.r, b1.r);
  mma_tf32(hi, a[0].h, a[1].h, a[2].h, a[3].h, b0.h, b1.h);
}
__device__ __forceinline__ uint32_t bits(float v) { return __float_as_uint(v); }
__device__ __forceinline__ float comp(const float4& v, int e) {
  return e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
}

// Four streamed values as parts.
__device__ __forceinline__ void read_parts(const float* y, uint4& h, uint4& r) {
  const float4 v = *reinterpret_cast<const float4*>(y);
  const Split a = split_inf(v.x), b = split_inf(v.y), c = split_inf(v.z), d = split_inf(v.w);
  h = make_uint4(a.h, b.h, c.h, d.h);
  r = make_uint4(a.r, b.r, c.r, d.r);
}

// s[nt] = 16 own rows (x) . 8 streamed rows (y)^T, summed over the
// channels.
template <typename C, bool kBf16>
__device__ __forceinline__ void scores(const float* x, const float* y, float (&s)[C::NT][4]) {
  const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  float lo[C::NT][4];
#pragma unroll
  for (int n = 0; n < C::NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[n][e] = lo[n][e] = 0.f;
#pragma unroll(C::DP == 64 ? 1 : 2)
  for (int bj = 0; bj < 2 * C::NB; ++bj) {
    const int d = 32 * (bj / 2) + 8 * t + 4 * (bj % 2);
    const float4 x0 = *reinterpret_cast<const float4*>(x + g * C::DPP + d);
    const float4 x1 = *reinterpret_cast<const float4*>(x + (g + 8) * C::DPP + d);
    if constexpr (kBf16) {
#pragma unroll
      for (int n = 0; n < C::NT; ++n) {
        const float4 v = *reinterpret_cast<const float4*>(y + (8 * n + g) * C::DPP + d);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          mma_tf32(s[n], bits(comp(x0, 2 * h)), bits(comp(x1, 2 * h)), bits(comp(x0, 2 * h + 1)),
                   bits(comp(x1, 2 * h + 1)), bits(comp(v, 2 * h)), bits(comp(v, 2 * h + 1)));
      }
    } else {
      Split a[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        a[h][0] = split(comp(x0, 2 * h));
        a[h][1] = split(comp(x1, 2 * h));
        a[h][2] = split(comp(x0, 2 * h + 1));
        a[h][3] = split(comp(x1, 2 * h + 1));
      }
#pragma unroll
      for (int n = 0; n < C::NT; ++n) {
        uint4 yh, yr;
        read_parts(y + (8 * n + g) * C::DPP + d, yh, yr);
        mma3(s[n], lo[n], a[0], {yh.x, yr.x}, {yh.y, yr.y});
        mma3(s[n], lo[n], a[1], {yh.z, yr.z}, {yh.w, yr.w});
      }
    }
  }
#pragma unroll
  for (int n = 0; n < C::NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[n][e] += lo[n][e];   // (bf16: zero)
}

// o += p (16 own rows x BS, as scores() leaves them) . y (BS streamed rows).
// Lane (g, t) holds, of rows g (elements 0, 1) and g + 8 (2, 3), channels 32 b + 8 t + e in
// o[4 b + e][0 or 2] and 32 b + 8 t + 4 + e in o[4 b + e][1 or 3].
template <typename C, bool kBf16>
__device__ __forceinline__ void add_values(const float (&p)[C::NT][4], const float* y,
                                           float (&o)[4 * C::NB][4]) {
  const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  Split a[C::NT][4];
#pragma unroll
  for (int n = 0; n < C::NT; ++n) {
    a[n][0] = split(p[n][0]);
    a[n][1] = split(p[n][2]);
    a[n][2] = split(p[n][1]);
    a[n][3] = split(p[n][3]);
  }
#pragma unroll
  for (int blk = 0; blk < C::NB; ++blk) {
    float hi[4][4], lo[4][4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int k = 0; k < 4; ++k) hi[e][k] = lo[e][k] = 0.f;
#pragma unroll
    for (int n = 0; n < C::NT; ++n) {
      const float* row = y + (8 * n + 2 * t) * C::DPP + 32 * blk + 4 * g;
      if constexpr (kBf16) {
        const float4 y0 = *reinterpret_cast<const float4*>(row), y1 = *reinterpret_cast<const float4*>(row + C::DPP);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          mma_tf32(lo[e], a[n][0].r, a[n][1].r, a[n][2].r, a[n][3].r, bits(comp(y0, e)), bits(comp(y1, e)));
          mma_tf32(hi[e], a[n][0].h, a[n][1].h, a[n][2].h, a[n][3].h, bits(comp(y0, e)), bits(comp(y1, e)));
        }
      } else {
        uint4 h0, h1, r0, r1;
        read_parts(row, h0, r0);
        read_parts(row + C::DPP, h1, r1);
        mma3(hi[0], lo[0], a[n], {h0.x, r0.x}, {h1.x, r1.x});
        mma3(hi[1], lo[1], a[n], {h0.y, r0.y}, {h1.y, r1.y});
        mma3(hi[2], lo[2], a[n], {h0.z, r0.z}, {h1.z, r1.z});
        mma3(hi[3], lo[3], a[n], {h0.w, r0.w}, {h1.w, r1.w});
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[4 * blk + e][k] += hi[e][k] + lo[e][k];
  }
}

// A later step's BS rows of one streamed tensor (fp32 rows of whole 16 bytes only), on their
// way to a buffer.
template <typename C, typename Off>
__device__ __forceinline__ void stage_tile(float* y, const float* src, int dim, Off off) {
  const int c0 = threadIdx.x % 16;
#pragma unroll
  for (int r = threadIdx.x / 16; r < C::BS; r += kF32Threads / 16) {
    const int64_t o = off(r);
#pragma unroll
    for (int c = c0; c < C::DP / 4; c += 16) {
      const bool real = o >= 0 && 4 * c < dim;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                       tc::smem_u32(y + r * C::DPP + 4 * c)),
                   "l"(reinterpret_cast<uint64_t>(real ? src + o + 4 * c : src)), "r"(real ? 16 : 0)
                   : "memory");
    }
  }
}

// N rows x dim of global memory -> shared, zeros past dim and where `off` gives none
// (negative).  16 threads per row, four channels at a time.
template <typename T, typename C, int N, typename Off>
__device__ __forceinline__ void load_tile(float* dst, const T* src, int dim, bool vec, Off off) {
  const int c0 = threadIdx.x % 16;
#pragma unroll 4
  for (int r = threadIdx.x / 16; r < N; r += kF32Threads / 16) {
    const int64_t o = off(r);
    const T* p = src + o;
#pragma unroll
    for (int c = c0; c < C::DP / 4; c += 16) {
      const int d = 4 * c;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (o >= 0 && d < dim) {
        if (sizeof(T) == 4 && vec) {
          v = *reinterpret_cast<const float4*>(p + d);
        } else if (vec) {
          const uint2 w = *reinterpret_cast<const uint2*>(p + d);
          v = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                          __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
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
// A block's source of keys: offsets of row r of the tile at key0, negative where the key is
// not permitted.
struct Keys {
  const Args& a;
  int b, len;
  int64_t kb, vb;
  __device__ Keys(const Args& a_, int b_, int hk, int len_)
      : a(a_), b(b_), len(len_), kb(b_ * a_.ks[0] + hk * a_.ks[2]), vb(b_ * a_.vs[0] + hk * a_.vs[2]) {}
  __device__ __forceinline__ int64_t k(int key) const { return key_ok(a, b, len, key) ? kb + (int64_t)key * a.ks[1] : -1; }
  __device__ __forceinline__ int64_t v(int key) const { return key_ok(a, b, len, key) ? vb + (int64_t)key * a.vs[1] : -1; }
};
// N keys from key0 of k and v, zeros where a key is not permitted; oks[r]: whether it is.
template <typename T, typename C, int N>
__device__ __forceinline__ void load_keys(const Keys& src, float* Ks, float* Vs, int* oks, int key0) {
  const Args& a = src.a;
  load_tile<T, C, N>(Ks, static_cast<const T*>(a.k), a.dim, a.vec, [&](int r) -> int64_t {
    const int64_t o = src.k(key0 + r);
    if (threadIdx.x % 16 == 0) oks[r] = o >= 0;
    return o;
  });
  load_tile<T, C, N>(Vs, static_cast<const T*>(a.v), a.dim, a.vec,
                     [&](int r) -> int64_t { return src.v(key0 + r); });
}
// The same for one streamed tile of fp32 rows, on its way.
template <typename C>
__device__ __forceinline__ void stage_keys(const Keys& src, float* y, int* ok, int key0) {
  const Args& a = src.a;
  stage_tile<C>(y, static_cast<const float*>(a.k), a.dim, [&](int r) {
    const int64_t o = src.k(key0 + r);
    if (threadIdx.x % 16 == 0) ok[r] = o >= 0;
    return o;
  });
  stage_tile<C>(y + C::TILE, static_cast<const float*>(a.v), a.dim, [&](int r) { return src.v(key0 + r); });
}
// The same of q and dO (rows of key head hk).
template <typename T, typename C, int N>
__device__ __forceinline__ void load_queries(const Args& a, float* Qs, float* Os, int b, int hk, int r0) {
  load_tile<T, C, N>(Qs, static_cast<const T*>(a.q), a.dim, a.vec, [&](int r) -> int64_t {
    return r0 + r < a.rows ? row_offset(a, a.qs, b, hk, r0 + r) : -1;
  });
  if (Os)
    load_tile<T, C, N>(Os, static_cast<const T*>(a.dout), a.dim, a.vec, [&](int r) -> int64_t {
      return r0 + r < a.rows ? row_offset(a, a.dos, b, hk, r0 + r) : -1;
    });
}
__device__ __forceinline__ void copy4(float* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc::smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ void staged() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// One of a lane's two rows (h = 0: g, 1: g + 8) of a result, to a row of T's or of fp32 parts.
template <typename C, typename T>
__device__ __forceinline__ void store_result(T* dst, const float (&o)[4 * C::NB][4], int h, int dim,
                                             float f) {
  const int t = threadIdx.x % 4;
#pragma unroll
  for (int b = 0; b < C::NB; ++b)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = 32 * b + 8 * t + 4 * i + e;
        if (d < dim) dst[d] = (T)(o[4 * b + e][2 * h + i] * f);
      }
}
template <typename C>
__device__ __forceinline__ void clear(float (&o)[4 * C::NB][4]) {
#pragma unroll
  for (int i = 0; i < 4 * C::NB; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(kAll, v, 1));
  return fmaxf(v, __shfl_xor_sync(kAll, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(kAll, v, 1);
  return v + __shfl_xor_sync(kAll, v, 2);
}

// grid: (row tiles x splits, kv_heads, batch)
template <typename T, typename C>
__global__ void __launch_bounds__(kF32Threads, C::DP <= 64 ? 4 : 2) f32_forward_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Y = Qs + kRows * C::DPP;        // K and V, two buffers
  int* oks = reinterpret_cast<int*>(Y + 4 * C::TILE);   // two buffers
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int split_id = blockIdx.x % a.splits, r0 = (int)(blockIdx.x / a.splits) * kRows;
  const int hk = blockIdx.y, b = blockIdx.z;
  const int len = walk_end(a, b);
  const int tiles = (len + C::BS - 1) / C::BS;
  const int t0 = (int)((int64_t)tiles * split_id / a.splits);
  const int t1 = (int)((int64_t)tiles * (split_id + 1) / a.splits);
  const Keys keys(a, b, hk, len);
  const bool async = sizeof(T) == 4 && a.vec;
  auto fetch = [&](int tile) {   // its keys, on their way to the buffer of its parity
    float* y = Y + tile % 2 * 2 * C::TILE;
    int* ok = oks + tile % 2 * C::BS;
    if (async) stage_keys<C>(keys, y, ok, tile * C::BS);
    else load_keys<T, C, C::BS>(keys, y, y + C::TILE, ok, tile * C::BS);
  };
  if (t0 < t1) fetch(t0);
  load_queries<T, C, kRows>(a, Qs, nullptr, b, hk, r0);
  const bool active = r0 + 16 * warp < a.rows;   // a warp without rows only loads
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[4 * C::NB][4];
  clear<C>(o);
  const float c2 = a.scale * kLog2e;
  for (int tile = t0; tile < t1; ++tile) {
    const float* Ks = Y + tile % 2 * 2 * C::TILE;
    const int* ok = oks + tile % 2 * C::BS;
    staged();
    __syncthreads();   // the tile is there, the other buffer is free
    if (tile + 1 < t1) fetch(tile + 1);
    if (!active) continue;
    float s[C::NT][4];
    scores<C, sizeof(T) == 2>(Qs + 16 * warp * C::DPP, Ks, s);
#pragma unroll
    for (int n = 0; n < C::NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = ok[8 * n + 2 * t + e % 2] ? s[n][e] * c2 : -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float top = m[h];
#pragma unroll
      for (int n = 0; n < C::NT; ++n) top = fmaxf(top, fmaxf(s[n][2 * h], s[n][2 * h + 1]));
      top = quad_max(top);
      const float base = top == -INFINITY ? 0.f : top;   // nothing permitted so far
      const float f = exp2f(m[h] - base);
      m[h] = top;
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < C::NT; ++n)
#pragma unroll
        for (int e = 2 * h; e < 2 * h + 2; ++e) {
          s[n][e] = exp2f(s[n][e] - base);
          sum += s[n][e];
        }
      l[h] = l[h] * f + sum;   // of this lane's columns
#pragma unroll
      for (int i = 0; i < 4 * C::NB; ++i) {
        o[i][2 * h] *= f;
        o[i][2 * h + 1] *= f;
      }
    }
    add_values<C, sizeof(T) == 2>(s, Ks + C::TILE, o);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] = quad_sum(l[h]);
    const int r = r0 + 16 * warp + g + 8 * h;
    if (r >= a.rows) continue;
    const float inv = l[h] > 0.f ? 1.f / l[h] : (l[h] == 0.f ? 0.f : l[h]);
    const float lse = l[h] == 0.f ? -INFINITY : m[h] * kLn2 + logf(l[h]);
    const int64_t row = ((int64_t)b * a.kv_heads + hk) * a.rows + r;
    const int64_t at = (int64_t)split_id * a.batch * a.kv_heads * a.rows + row;
    if (a.splits == 1) {
      store_result<C>(static_cast<T*>(a.out) + row_offset(a, a.os, b, hk, r), o, h, a.dim, inv);
      if (a.lse && t == 0) a.lse[row] = lse;
    } else {
      store_result<C>(a.part_o + at * a.dim, o, h, a.dim, inv);
      if (t == 0) a.part_lse[at] = lse;
    }
  }
}

// grid: (key tiles x dkv_splits + row tiles x dq_splits, kv_heads, batch); the first
// produce dK and dV (own rows: keys; streamed: queries), the others dQ (the reverse).
template <typename T, typename C>
__global__ void __launch_bounds__(kF32Threads, C::DP <= 64 ? 3 : 2) f32_backward_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) float sm[];
  float* X0 = sm;                        // own: K or Q
  float* X1 = X0 + kRows * C::DPP;       //      V or dO
  float* Y = X1 + kRows * C::DPP;        // streamed, two buffers: Q and dO, or K and V
  float* stats = Y + 4 * C::TILE;        // dK/dV, two buffers: lse, delta of those queries
  int* oks = reinterpret_cast<int*>(stats + 4 * C::BS);   // own keys, or two buffers of streamed ones
  static_assert(kRows >= 2 * C::BS, "");
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int hk = blockIdx.y, b = blockIdx.z;
  const int len = walk_end(a, b);
  const int dkv_blocks = (a.len_kv + kRows - 1) / kRows * a.dkv_splits;
  const float c2 = a.scale * kLog2e;
  const float* lse_row = a.lse_in + ((int64_t)b * a.kv_heads + hk) * a.rows;
  const float* delta_row = a.delta + ((int64_t)b * a.kv_heads + hk) * a.rows;
  // past the rows, or a row without keys: P = exp(S - inf) = 0
  auto base2 = [&](float lse, bool real) { return real && lse != -INFINITY ? lse * kLog2e : INFINITY; };
  const bool async = sizeof(T) == 4 && a.vec;
  const float *x0 = X0 + 16 * warp * C::DPP, *x1 = X1 + 16 * warp * C::DPP;
  float p[C::NT][4], ds[C::NT][4];
  const Keys keys(a, b, hk, len);
  if ((int)blockIdx.x < dkv_blocks) {   // ----------------------------- dK, dV
    const int k0 = (int)blockIdx.x / a.dkv_splits * kRows, part = (int)blockIdx.x % a.dkv_splits;
    const int steps = (a.rows + C::BS - 1) / C::BS;
    const int s0 = (int)((int64_t)steps * part / a.dkv_splits);
    const int s1 = (int)((int64_t)steps * (part + 1) / a.dkv_splits);
    float dk[4 * C::NB][4], dv[4 * C::NB][4];
    clear<C>(dk);
    clear<C>(dv);
    if (k0 < len) {
      auto fetch = [&](int step) {   // its queries, on their way to the buffer of its parity
        const int r0 = step * C::BS;
        float *y = Y + step % 2 * 2 * C::TILE, *st = stats + step % 2 * 2 * C::BS;
        if (async) {
          stage_tile<C>(y, static_cast<const float*>(a.q), a.dim, [&](int r) -> int64_t {
            return r0 + r < a.rows ? row_offset(a, a.qs, b, hk, r0 + r) : -1;
          });
          stage_tile<C>(y + C::TILE, static_cast<const float*>(a.dout), a.dim, [&](int r) -> int64_t {
            return r0 + r < a.rows ? row_offset(a, a.dos, b, hk, r0 + r) : -1;
          });
        } else {
          load_queries<T, C, C::BS>(a, y, y + C::TILE, b, hk, r0);
        }
        if (threadIdx.x < 2 * C::BS) {
          const int r = r0 + threadIdx.x % C::BS;
          copy4(st + threadIdx.x, (threadIdx.x < C::BS ? lse_row : delta_row) + min(r, a.rows - 1));
        }
      };
      if (s0 < s1) fetch(s0);
      load_keys<T, C, kRows>(keys, X0, X1, oks, k0);
      __syncthreads();
      for (int step = s0; step < s1; ++step) {
        const int r0 = step * C::BS;
        const float *Y0 = Y + step % 2 * 2 * C::TILE, *Y1 = Y0 + C::TILE, *st = stats + step % 2 * 2 * C::BS;
        staged();
        __syncthreads();   // the tile is there, the other buffer is free
        if (step + 1 < s1) fetch(step + 1);
        if (k0 + 16 * warp >= len) continue;
        // (a key that is not permitted has zero rows of K and V; its results are dropped
        // below)
        scores<C, sizeof(T) == 2>(x0, Y0, p);
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int q = 8 * n + 2 * t + e % 2;
            p[n][e] = exp2f(fmaf(p[n][e], c2, -base2(st[q], r0 + q < a.rows)));
          }
        add_values<C, sizeof(T) == 2>(p, Y1, dv);   // (before dP: its registers are free here)
        scores<C, sizeof(T) == 2>(x1, Y1, ds);
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) ds[n][e] = p[n][e] * (ds[n][e] - st[C::BS + 8 * n + 2 * t + e % 2]);
        add_values<C, sizeof(T) == 2>(ds, Y0, dk);
      }
    }
    if (one_key(a, b, len)) clear<C>(dk);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int own = 16 * warp + g + 8 * h, key = k0 + own;
      if (key >= a.len_kv) continue;
      if (k0 >= len || !oks[own])
#pragma unroll
        for (int i = 0; i < 4 * C::NB; ++i)
#pragma unroll
          for (int e = 2 * h; e < 2 * h + 2; ++e) dk[i][e] = dv[i][e] = 0.f;
      if (a.dkv_splits == 1) {
        store_result<C>(static_cast<T*>(a.dk) + b * a.dks[0] + key * a.dks[1] + hk * a.dks[2], dk, h, a.dim, a.scale);
        store_result<C>(static_cast<T*>(a.dv) + b * a.dvs[0] + key * a.dvs[1] + hk * a.dvs[2], dv, h, a.dim, 1.f);
      } else {
        const int64_t at = ((((int64_t)part * a.batch + b) * a.kv_heads + hk) * a.len_kv + key) * a.dim;
        store_result<C>(a.part_dk + at, dk, h, a.dim, 1.f);
        store_result<C>(a.part_dv + at, dv, h, a.dim, 1.f);
      }
    }
    return;
  }
  // ---------------------------------------------------------------------- dQ
  const int id = (int)blockIdx.x - dkv_blocks;
  const int r0 = id / a.dq_splits * kRows, part = id % a.dq_splits;
  const int steps = (len + C::BS - 1) / C::BS;
  const int s0 = (int)((int64_t)steps * part / a.dq_splits);
  const int s1 = (int)((int64_t)steps * (part + 1) / a.dq_splits);
  float dq[4 * C::NB][4];
  clear<C>(dq);
  auto fetch = [&](int step) {   // its keys, on their way to the buffer of its parity
    const int k0 = step * C::BS;
    float* y = Y + step % 2 * 2 * C::TILE;
    int* ok = oks + step % 2 * C::BS;
    if (async) {
      stage_keys<C>(keys, y, ok, k0);
    } else {
      load_keys<T, C, C::BS>(keys, y, y + C::TILE, ok, k0);
    }
  };
  if (s0 < s1) fetch(s0);
  load_queries<T, C, kRows>(a, X0, X1, b, hk, r0);
  const bool active = r0 + 16 * warp < a.rows;
  float lse[2], delta[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = r0 + 16 * warp + g + 8 * h;
    lse[h] = base2(r < a.rows ? lse_row[r] : 0.f, r < a.rows);
    delta[h] = r < a.rows ? delta_row[r] : 0.f;
  }
  for (int step = s0; step < s1; ++step) {
    const float *Y0 = Y + step % 2 * 2 * C::TILE, *Y1 = Y0 + C::TILE;
    const int* ok = oks + step % 2 * C::BS;
    staged();
    __syncthreads();
    if (step + 1 < s1) fetch(step + 1);
    if (!active) continue;
    scores<C, sizeof(T) == 2>(x0, Y0, p);
    scores<C, sizeof(T) == 2>(x1, Y1, ds);
#pragma unroll
    for (int n = 0; n < C::NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        ds[n][e] = ok[8 * n + 2 * t + e % 2]
                       ? exp2f(fmaf(p[n][e], c2, -lse[e / 2])) * (ds[n][e] - delta[e / 2])
                       : 0.f;
    add_values<C, sizeof(T) == 2>(ds, Y0, dq);
  }
  if (one_key(a, b, len)) clear<C>(dq);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = r0 + 16 * warp + g + 8 * h;
    if (r >= a.rows) continue;
    if (a.dq_splits == 1) {
      store_result<C>(static_cast<T*>(a.dq) + row_offset(a, a.dqs, b, hk, r), dq, h, a.dim, a.scale);
    } else {
      const int64_t at = ((((int64_t)part * a.batch + b) * a.kv_heads + hk) * a.rows + r) * a.dim;
      store_result<C>(a.part_dq + at, dq, h, a.dim, 1.f);
    }
  }
}

// delta of bf16 inputs where at most kExactKeys keys are permitted (sum_d dout out would carry
// out's rounding into every dS): the first half of a dQ block.  grid: (row tiles, kv_heads,
// batch)
template <typename T, typename C>
__global__ void __launch_bounds__(kF32Threads) f32_delta_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) float sm[];
  float* X0 = sm;
  float* X1 = X0 + kRows * C::DPP;
  float* Y0 = X1 + kRows * C::DPP;
  float* Y1 = Y0 + C::TILE;
  int* oks = reinterpret_cast<int*>(Y1 + C::TILE);
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int hk = blockIdx.y, b = blockIdx.z, r0 = blockIdx.x * kRows;
  const int len = walk_end(a, b);
  int count = len;   // permitted keys, as far as it matters
  if (a.key_mask && len > kExactKeys) {
    count = 0;
    for (int key0 = 0; key0 < len && count <= kExactKeys; key0 += 512) {
      int mine = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) mine += key_ok(a, b, len, key0 + 32 * i + lane);
      count += __reduce_add_sync(kAll, mine);
    }
  }
  if (count > kExactKeys) return;   // as delta_kernel took it from out
  const float c2 = a.scale * kLog2e;
  const int64_t row0 = ((int64_t)b * a.kv_heads + hk) * a.rows;
  load_queries<T, C, kRows>(a, X0, X1, b, hk, r0);
  float lse2[2], sum[2] = {0.f, 0.f};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = r0 + 16 * warp + g + 8 * h;
    lse2[h] = r < a.rows ? a.lse_in[row0 + r] * kLog2e : INFINITY;
  }
  const Keys keys(a, b, hk, len);
  for (int k0 = 0; k0 < len; k0 += C::BS) {
    __syncthreads();
    load_keys<T, C, C::BS>(keys, Y0, Y1, oks, k0);
    __syncthreads();
    float p[C::NT][4], dp[C::NT][4];
    scores<C, sizeof(T) == 2>(X0 + 16 * warp * C::DPP, Y0, p);
    scores<C, sizeof(T) == 2>(X1 + 16 * warp * C::DPP, Y1, dp);
#pragma unroll
    for (int n = 0; n < C::NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (oks[8 * n + 2 * t + e % 2])
          sum[e / 2] = fmaf(exp2f(fmaf(p[n][e], c2, -lse2[e / 2])), dp[n][e], sum[e / 2]);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float d = quad_sum(sum[h]);
    const int r = r0 + 16 * warp + g + 8 * h;
    if (t == 0 && r < a.rows) a.delta[row0 + r] = d;
  }
}

template <typename T, typename C>
kfac_status launch_forward(const Args& a, cudaStream_t st) {
  static OncePerDevice once;
  const kfac_status e = allow_smem(once, f32_forward_kernel<T, C>, C::FWD);
  if (e != KFAC_OK) return e;
  const dim3 grid((unsigned)(cdiv(a.rows, kRows) * a.splits), a.kv_heads, a.batch);
  launch_pdl(f32_forward_kernel<T, C>, grid, dim3(kF32Threads), C::FWD, st, a);
  count_launch();
  return check_launch();
}
template <typename T, typename C>
kfac_status launch_backward(const Args& a, cudaStream_t st) {
  static OncePerDevice once;
  const kfac_status e = allow_smem(once, f32_backward_kernel<T, C>, C::BWD);
  if (e != KFAC_OK) return e;
  const dim3 grid((unsigned)(cdiv(a.len_kv, kRows) * a.dkv_splits + cdiv(a.rows, kRows) * a.dq_splits),
                  a.kv_heads, a.batch);
  launch_pdl(f32_backward_kernel<T, C>, grid, dim3(kF32Threads), C::BWD, st, a);
  count_launch();
  return check_launch();
}

template <typename C>
kfac_status launch_delta(const Args& a, cudaStream_t st) {
  static OncePerDevice once;
  const kfac_status e = allow_smem(once, f32_delta_kernel<__nv_bfloat16, C>, C::BWD);
  if (e != KFAC_OK) return e;
  launch_pdl(f32_delta_kernel<__nv_bfloat16, C>, dim3((unsigned)cdiv(a.rows, kRows), a.kv_heads, a.batch),
             dim3(kF32Threads), C::BWD, st, a);
  count_launch();
  return check_launch();
}

}  // namespace

// Tiles as long as the registers of 4 (128 channels: 2) and 3 (2) blocks per SM allow;
// backward with 32 channels: 430 us in tiles of 16 and 440 in tiles of 32; with 64, 777 and 735.
// The blocks per SM are worth their spills (up to 76 bytes a thread forward, 88 backward; bf16
// rows 100 and 280).  4 x 1024 x 1024, 8 heads, us with 4 and 3 blocks forward: 64 channels 218,
// 232; 32: 132, 153; 36 in bf16: 203, 355; with 3 and 2 backward: 742, 769; 439, 489; 576, 687.
template <typename T> kfac_status f32_forward(const Args& a, cudaStream_t st) {
  if (a.dim <= 32) return launch_forward<T, Cfg<64, 32>>(a, st);
  return a.dim <= 64 ? launch_forward<T, Cfg<32, 64>>(a, st) : launch_forward<T, Cfg<32, 128>>(a, st);
}
template <typename T> kfac_status f32_backward(const Args& a, cudaStream_t st) {
  if (a.dim <= 32) return launch_backward<T, Cfg<16, 32>>(a, st);
  return a.dim <= 64 ? launch_backward<T, Cfg<32, 64>>(a, st) : launch_backward<T, Cfg<16, 128>>(a, st);
}
kfac_status f32_delta(const Args& a, cudaStream_t st) {
  return a.dim <= 64 ? launch_delta<Cfg<32, 64>>(a, st) : launch_delta<Cfg<16, 128>>(a, st);
}
template kfac_status f32_forward<float>(const Args&, cudaStream_t);
template kfac_status f32_forward<__nv_bfloat16>(const Args&, cudaStream_t);
template kfac_status f32_backward<float>(const Args&, cudaStream_t);
template kfac_status f32_backward<__nv_bfloat16>(const Args&, cudaStream_t);

}  // namespace attn
}  // namespace kfac
