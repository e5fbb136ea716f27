// Cross attention of few query rows (bf16): single new tokens against long encoder
// states.  rows = heads of a group x queries, 16 of them per block.
//
// Bound by memory: k and v are read once, at about 4 flop per byte and row.  A warp
// takes 16 keys at a time straight from memory into the fragments of mma.sync
// m16n8k16 - no shared memory, no barriers in the loop.  The order of channels within
// a product is free as long as both operands agree, and so is the order of keys in
// P V, so every lane loads whole 16-byte pieces:
//   k: lane (g, t) = (lane / 4, lane % 4) takes key g (and 8 + g), channels
//      32 c + 8 t .. + 7: two k-steps of S = q k^T;
//   v: keys 2t, 2t + 1, 8 + 2t, 8 + 2t + 1 (the columns of S this lane holds),
//      channels 64 c + 8 g .. + 7; pairs of keys interleave into eight n-tiles of P V.
// P enters as two bf16 parts (high and remainder): the second product costs nothing
// here and keeps P exact to 2^-17.
// Blocks take fixed lengths of the key axis (many more than fit at once, so that
// ragged lengths balance); parts are joined by the combine kernel.
#include "attn.cuh"

namespace kfac {
namespace attn {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// (hi, lo) bf16 pairs of two fp32 values
__device__ __forceinline__ void split2(float x, float y, uint32_t* hi, uint32_t* lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  const __nv_bfloat162 l = __floats2bfloat162_rn(x - __bfloat162float(h.x), y - __bfloat162float(h.y));
  *hi = *reinterpret_cast<const uint32_t*>(&h);
  *lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) {
  uint4 v;   // read once: keep it out of L1
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(kFull, v, 1));
  return fmaxf(v, __shfl_xor_sync(kFull, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(kFull, v, 1);
  return v + __shfl_xor_sync(kFull, v, 2);
}

// DC: 32-channel pieces (dim <= 32 DC), VC: 64-channel pieces.
// grid: (16-row tiles x parts, kv_heads, batch); part s: keys [s, s + 1) x part_keys
template <int DC>
__global__ void __launch_bounds__(kTokenWarps * 32)
token_kernel(const __grid_constant__ Args a) {
  constexpr int VC = (DC + 1) / 2;
  __shared__ float so[kTokenWarps][16][32 * DC + 4];
  __shared__ float sm[kTokenWarps][16], sl[kTokenWarps][16];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int split = (int)(blockIdx.x % a.splits), r0 = (int)(blockIdx.x / a.splits) * 16;
  const int hk = blockIdx.y, b = blockIdx.z;
  const int len = key_count(a, b);
  const int first = split * a.part_keys, last = min(len, first + a.part_keys);
  const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(a.k) + b * a.ks[0] + hk * a.ks[2];
  const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(a.v) + b * a.vs[0] + hk * a.vs[2];

  uint4 kr[2][DC], vr[4][VC];
  bool ok[4];
  auto load_k = [&](int key0) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < DC; ++c) {
        const int key = key0 + 8 * i + g, d = 32 * c + 8 * t;
        kr[i][c] = make_uint4(0, 0, 0, 0);
        if (key < last && d < a.dim) kr[i][c] = load16(kp + key * a.ks[1] + d);
      }
  };
  auto load_v = [&](int key0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = key0 + (i / 2) * 8 + 2 * t + i % 2;
      ok[i] = key < last && (!a.key_mask || __ldg(a.key_mask + (int64_t)b * a.len_kv + key) != 0);
#pragma unroll
      for (int c = 0; c < VC; ++c) {
        const int d = 64 * c + 8 * g;
        vr[i][c] = make_uint4(0, 0, 0, 0);   // not permitted: whatever is there stays out
        if (ok[i] && d < a.dim) vr[i][c] = load16(vp + key * a.vs[1] + d);
      }
    }
  };

  int key0 = first + 16 * warp;
  if (key0 < last) load_k(key0);
  // rows g and g + 8 of q, as A fragments
  uint4 qr[2][DC];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + 8 * i + g;
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) +
                              (r < a.rows ? row_offset(a, a.qs, b, hk, r) : 0);
#pragma unroll
    for (int c = 0; c < DC; ++c) {
      qr[i][c] = make_uint4(0, 0, 0, 0);
      if (r < a.rows && 32 * c + 8 * t < a.dim)
        qr[i][c] = *reinterpret_cast<const uint4*>(qp + 32 * c + 8 * t);
    }
  }
  if (key0 < last) load_v(key0);
  const float c2 = a.scale * kLog2e;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[VC][8][4];
#pragma unroll
  for (int c = 0; c < VC; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][j][e] = 0.f;

  for (; key0 < last; key0 += 16 * kTokenWarps) {
    const int next = key0 + 16 * kTokenWarps;
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int c = 0; c < DC; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mma16816(s[i], qr[0][c].x, qr[1][c].x, qr[0][c].y, qr[1][c].y, kr[i][c].x, kr[i][c].y);
        mma16816(s[i], qr[0][c].z, qr[1][c].z, qr[0][c].w, qr[1][c].w, kr[i][c].z, kr[i][c].w);
      }
    if (next < last) load_k(next);
    // rows g (e = 0, 1) and g + 8 (e = 2, 3); columns 8 i + 2 t + e % 2
    float mn[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = ok[2 * i + e % 2] ? s[i][e] * c2 : -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      mn[h] = fmaxf(m[h], quad_max(fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]),
                                         fmaxf(s[1][2 * h], s[1][2 * h + 1]))));
    if (__any_sync(kFull, mn[0] > m[0] || mn[1] > m[1])) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float f = mn[h] == m[h] ? 1.f : exp2f(m[h] - mn[h]);
        m[h] = mn[h];
        l[h] *= f;
#pragma unroll
        for (int c = 0; c < VC; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            o[c][j][2 * h] *= f;
            o[c][j][2 * h + 1] *= f;
          }
      }
    }
    uint32_t hi[4], lo[4];   // A fragments: (row g, tile 0), (g + 8, 0), (g, 1), (g + 8, 1)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float base = m[h] == -INFINITY ? 0.f : m[h];
        const float x = exp2f(s[i][2 * h] - base), y = exp2f(s[i][2 * h + 1] - base);
        l[h] += x + y;
        split2(x, y, &hi[2 * i + h], &lo[2 * i + h]);
      }
#pragma unroll
    for (int c = 0; c < VC; ++c) {
      const uint32_t w[4][4] = {{vr[0][c].x, vr[0][c].y, vr[0][c].z, vr[0][c].w},
                                {vr[1][c].x, vr[1][c].y, vr[1][c].z, vr[1][c].w},
                                {vr[2][c].x, vr[2][c].y, vr[2][c].z, vr[2][c].w},
                                {vr[3][c].x, vr[3][c].y, vr[3][c].z, vr[3][c].w}};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t sel = j % 2 ? 0x7632u : 0x5410u;
        const uint32_t b0 = __byte_perm(w[0][j / 2], w[1][j / 2], sel);
        const uint32_t b1 = __byte_perm(w[2][j / 2], w[3][j / 2], sel);
        mma16816(o[c][j], hi[0], hi[1], hi[2], hi[3], b0, b1);
        mma16816(o[c][j], lo[0], lo[1], lo[2], lo[3], b0, b1);
      }
    }
    if (next < last) load_v(next);
  }

  // join the warps: each row's largest maximum, sums rescaled to it
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] = quad_sum(l[h]);
    if (t == 0) {
      sm[warp][g + 8 * h] = m[h];
      sl[warp][g + 8 * h] = l[h];
    }
#pragma unroll
    for (int c = 0; c < VC; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int d = 64 * c + 8 * (2 * t + e) + j;
          if (d < 32 * DC) so[warp][g + 8 * h][d] = o[c][j][2 * h + e];
        }
  }
  __syncthreads();
  const int rows = min(16, a.rows - r0);
  for (int r = warp; r < rows; r += kTokenWarps) {
    float top = -INFINITY, total = 0.f, f[kTokenWarps];
#pragma unroll
    for (int w = 0; w < kTokenWarps; ++w) top = fmaxf(top, sm[w][r]);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < kTokenWarps; ++w) {
      f[w] = exp2f(sm[w][r] - base);
      total += f[w] * sl[w][r];
    }
    const float inv = total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);
    const float lse = total == 0.f ? -INFINITY : (base + log2f(total)) * kLn2;
    const int64_t row = ((int64_t)b * a.kv_heads + hk) * a.rows + r0 + r;
    const int64_t part = (int64_t)split * a.batch * a.kv_heads * a.rows + row;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + row_offset(a, a.os, b, hk, r0 + r);
    for (int d = lane; d < a.dim; d += 32) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kTokenWarps; ++w) v = fmaf(f[w], so[w][r][d], v);
      if (a.splits == 1) dst[d] = __float2bfloat16_rn(v * inv);
      else a.part_o[part * a.dim + d] = v * inv;
    }
    if (lane == 0) {
      if (a.splits > 1) a.part_lse[part] = lse;
      else if (a.lse) a.lse[row] = lse;
    }
  }
}

}  // namespace

kfac_status token_forward(const Args& a, cudaStream_t st) {
  const dim3 grid((unsigned)(cdiv(a.rows, 16) * a.splits), a.kv_heads, a.batch), block(kTokenWarps * 32);
  if (a.dim <= 32) launch_pdl(token_kernel<1>, grid, block, 0, st, a);
  else if (a.dim <= 64) launch_pdl(token_kernel<2>, grid, block, 0, st, a);
  else if (a.dim <= 96) launch_pdl(token_kernel<3>, grid, block, 0, st, a);
  else launch_pdl(token_kernel<4>, grid, block, 0, st, a);
  count_launch();
  return check_launch();
}

}  // namespace attn
}  // namespace kfac
