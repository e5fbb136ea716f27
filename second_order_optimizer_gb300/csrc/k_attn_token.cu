// Cross attention of few query rows (bf16): single new tokens against long encoder
// states.  rows = heads of a group x queries, 16 of them per block.
//
// Bound by memory: k and v are read once, at 2 flop per byte and row.  Each warp walks
// 16 keys at a time through a ring of its own in shared memory (16-byte cp.async, one
// step ahead, no block-wide barrier; 128 channels: 65 KB a block, three blocks per SM;
// two steps ahead and two blocks: a tenth more): S = q k^T and O += P v by mma.sync
// m16n8k16 on fragments that ldmatrix reads, rows swizzled so that eight rows of one
// 16-byte column hit all banks.  32 x 8192 keys on 4 key heads x 128, 16 heads: 84 us for
// 537 MB (6.4 TB/s), 50 us for ragged lengths (5.5 TB/s).  Keys that are not permitted are
// filled with zeros, their scores are -infinity.  P enters as two bf16 parts (high and
// remainder): the second product costs nothing here and keeps P exact to 2^-17.
//
// The key axis is split.  Up to 8 parts are the blocks of one cluster, each taking its
// share of the sequence's own length; they exchange maxima, sums and outputs through
// distributed shared memory and the call is one launch.  More parts (few sequences,
// long states) are fixed lengths of the axis, joined by the combine kernel.  Ragged lengths
// that fill more than one wave start with the longest, so that the short ones fill the end.
#include "attn.cuh"
#include "tc_prims.cuh"

namespace kfac {
namespace attn {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kStages = 2;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// 16 bytes, or zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// (hi, lo) bf16 pairs of two fp32 values
__device__ __forceinline__ void split2(float x, float y, uint32_t* hi, uint32_t* lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  const __nv_bfloat162 l = __floats2bfloat162_rn(x - __bfloat162float(h.x), y - __bfloat162float(h.y));
  *hi = *reinterpret_cast<const uint32_t*>(&h);
  *lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(kFull, v, 1));
  return fmaxf(v, __shfl_xor_sync(kFull, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(kFull, v, 1);
  return v + __shfl_xor_sync(kFull, v, 2);
}

template <int DC> struct TokenCfg {            // dim <= 32 DC
  static constexpr int CH = 4 * DC;            // 16-byte pieces per row
  static constexpr int ROW = 64 * DC;          // bytes
  static constexpr int TILE = 16 * ROW;        // 16 keys of k or of v
  static constexpr int RING = kStages * 2 * TILE;   // per warp
  static constexpr int OP = 32 * DC + 4;       // pitch of an output row (floats)
  static constexpr size_t JOIN = sizeof(float) * (kTokenWarps + 1) * (16 * OP + 32);
  static constexpr size_t SMEM = (size_t)kTokenWarps * RING > JOIN ? (size_t)kTokenWarps * RING : JOIN;
  __device__ static uint32_t at(int row, int chunk) {
    return (uint32_t)(row * ROW + ((chunk ^ (DC % 2 ? row >> 1 & 3 : row & 7)) << 4));
  }
};

// The batch entry that `rank` others precede when the longest come first (equal ones in
// their order).  A thread per entry, up to kTokenOrdered of them; whole blocks.
__device__ __forceinline__ int entry_by_length(const Args& a, int rank) {
  __shared__ int len[kTokenOrdered], entry;
  const int i = threadIdx.x, mine = i < a.batch ? key_count(a, i) : 0;
  len[i] = mine;
  __syncthreads();
  int before = 0;
  for (int j = 0; j < a.batch; ++j) before += len[j] > mine || (len[j] == mine && j < i);
  if (i < a.batch && before == rank) entry = i;
  __syncthreads();
  return entry;
}

// grid: (16-row tiles x parts, kv_heads, batch).  kCluster: a tile's parts are one
// cluster and share the sequence's length; otherwise part s takes keys
// [s, s + 1) x part_keys.
template <int DC, bool kCluster>
__global__ void __launch_bounds__(kTokenWarps * 32, kTokenPerSm)
token_kernel(const __grid_constant__ Args a) {
  using C = TokenCfg<DC>;
  extern __shared__ __align__(1024) uint8_t smem[];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int split = (int)(blockIdx.x % a.splits), r0 = (int)(blockIdx.x / a.splits) * 16;
  const int hk = blockIdx.y, b = a.longest_first ? entry_by_length(a, blockIdx.z) : blockIdx.z;
  const int len = walk_end(a, b);
  int first, last;
  if (kCluster) {
    const int blocks = (len + 15) / 16;
    first = (int)((int64_t)blocks * split / a.splits) * 16;
    last = min(len, (int)((int64_t)blocks * (split + 1) / a.splits) * 16);
  } else {
    first = split * a.part_keys;
    last = min(len, first + a.part_keys);
  }
  const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(a.k) + b * a.ks[0] + hk * a.ks[2];
  const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(a.v) + b * a.vs[0] + hk * a.vs[2];
  const uint8_t* mp = a.key_mask ? a.key_mask + (int64_t)b * a.len_kv : nullptr;
  const uint32_t ring = tc::smem_u32(smem) + warp * C::RING;
  const int begin = first + 16 * warp, step = 16 * kTokenWarps;

  // permitted keys among the 16 from key0 (bit i), given this lane's mask byte
  auto word = [&](int key0, uint8_t byte) {
    const int n = last - key0;
    const uint32_t w = n >= 16 ? 0xffffu : n <= 0 ? 0u : (1u << n) - 1u;
    return mp ? w & __ballot_sync(kFull, byte != 0) : w;
  };
  auto mask_byte = [&](int key0) -> uint8_t {
    const int key = key0 + lane;
    return mp && lane < 16 && key < last ? __ldg(mp + key) : (uint8_t)0;
  };
  auto fetch = [&](int key0, int stage, uint32_t w) {
    const uint32_t ks = ring + stage * 2 * C::TILE, vs = ks + C::TILE;
#pragma unroll
    for (int i = 0; i < 2 * DC; ++i) {
      const int e = lane + 32 * i, row = e / C::CH, c = e % C::CH;
      const bool real = (w >> row & 1u) && 8 * c < a.dim;
      copy16(ks + C::at(row, c), real ? kp + (key0 + row) * a.ks[1] + 8 * c : kp, real);
      copy16(vs + C::at(row, c), real ? vp + (key0 + row) * a.vs[1] + 8 * c : vp, real);
    }
  };

  uint32_t words[kStages];
#pragma unroll
  for (int s = 0; s + 1 < kStages; ++s) {
    const int key0 = begin + s * step;
    words[s] = word(key0, mask_byte(key0));
    if (key0 < last) fetch(key0, s, words[s]);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  uint8_t byte = mask_byte(begin + (kStages - 1) * step);

  // rows g and g + 8 of q, as A fragments
  uint32_t qr[2 * DC][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + 8 * i + g;
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) +
                              (r < a.rows ? row_offset(a, a.qs, b, hk, r) : 0);
#pragma unroll
    for (int kk = 0; kk < 2 * DC; ++kk)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int d = 16 * kk + 8 * e + 2 * t;
        qr[kk][2 * e + i] = r < a.rows && d < a.dim ? *reinterpret_cast<const uint32_t*>(qp + d) : 0u;
      }
  }
  const float c2 = a.scale * kLog2e;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[C::CH][4];
#pragma unroll
  for (int c = 0; c < C::CH; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[c][e] = 0.f;

  int stage = 0;
  for (int key0 = begin; key0 < last; key0 += step) {
    // the stage that the previous step has read takes the keys kStages - 1 steps ahead
    const int ahead = key0 + (kStages - 1) * step;
    words[kStages - 1] = word(ahead, byte);
    byte = mask_byte(ahead + step);
    __syncwarp();
    if (ahead < last) fetch(ahead, stage == 0 ? kStages - 1 : stage - 1, words[kStages - 1]);
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const uint32_t ks = ring + stage * 2 * C::TILE, vs = ks + C::TILE, w = words[0];
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int kk = 0; kk < 2 * DC; ++kk) {
      uint32_t f[4];
      ldm4(ks + C::at((lane / 16) * 8 + lane % 8, 2 * kk + lane / 8 % 2), f);
      mma16816(s[0], qr[kk][0], qr[kk][1], qr[kk][2], qr[kk][3], f[0], f[1]);
      mma16816(s[1], qr[kk][0], qr[kk][1], qr[kk][2], qr[kk][3], f[2], f[3]);
    }
    // rows g (e = 0, 1) and g + 8 (e = 2, 3); columns 8 i + 2 t + e % 2
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s[i][e] = w >> (8 * i + 2 * t + e % 2) & 1u ? s[i][e] * c2 : -INFINITY;
    float mn[2];
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
        for (int c = 0; c < C::CH; ++c) {
          o[c][2 * h] *= f;
          o[c][2 * h + 1] *= f;
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
    for (int c = 0; c < C::CH; c += 2) {
      uint32_t f[4];
      ldm4_t(vs + C::at(lane / 8 % 2 * 8 + lane % 8, c + lane / 16), f);
      mma16816(o[c], hi[0], hi[1], hi[2], hi[3], f[0], f[1]);
      mma16816(o[c + 1], hi[0], hi[1], hi[2], hi[3], f[2], f[3]);
      mma16816(o[c], lo[0], lo[1], lo[2], lo[3], f[0], f[1]);
      mma16816(o[c + 1], lo[0], lo[1], lo[2], lo[3], f[2], f[3]);
    }
#pragma unroll
    for (int i = 0; i + 1 < kStages; ++i) words[i] = words[i + 1];
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }

  // join the warps (the rings are free): each row's largest maximum, sums and outputs
  // rescaled to it, left in part [kTokenWarps]
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  constexpr int PART = 16 * C::OP + 32;   // floats: rows, then 16 maxima and 16 sums
  float* parts = reinterpret_cast<float*>(smem);
  float* mine = parts + warp * PART;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] = quad_sum(l[h]);
    if (t == 0) {
      mine[16 * C::OP + g + 8 * h] = m[h];
      mine[16 * C::OP + 16 + g + 8 * h] = l[h];
    }
#pragma unroll
    for (int c = 0; c < C::CH; ++c)
      *reinterpret_cast<float2*>(mine + (g + 8 * h) * C::OP + 8 * c + 2 * t) =
          make_float2(o[c][2 * h], o[c][2 * h + 1]);
  }
  __syncthreads();
  const int rows = min(16, a.rows - r0);
  float* all = parts + kTokenWarps * PART;
  for (int r = warp; r < rows; r += kTokenWarps) {
    float top = -INFINITY, total = 0.f, f[kTokenWarps];
#pragma unroll
    for (int w = 0; w < kTokenWarps; ++w) top = fmaxf(top, parts[w * PART + 16 * C::OP + r]);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < kTokenWarps; ++w) {
      f[w] = exp2f(parts[w * PART + 16 * C::OP + r] - base);
      total += f[w] * parts[w * PART + 16 * C::OP + 16 + r];
    }
    const float inv = total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);
    const float lse = total == 0.f ? -INFINITY : (base + log2f(total)) * kLn2;
    const int64_t row = ((int64_t)b * a.kv_heads + hk) * a.rows + r0 + r;
    const int64_t part = (int64_t)split * a.batch * a.kv_heads * a.rows + row;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + row_offset(a, a.os, b, hk, r0 + r);
    for (int d = lane; d < a.dim; d += 32) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kTokenWarps; ++w) v = fmaf(f[w], parts[w * PART + r * C::OP + d], v);
      if (kCluster) all[r * C::OP + d] = v;
      else if (a.splits == 1) dst[d] = __float2bfloat16_rn(v * inv);
      else a.part_o[part * a.dim + d] = v * inv;
    }
    if (lane == 0) {
      if (kCluster) {
        all[16 * C::OP + r] = top;
        all[16 * C::OP + 16 + r] = total;
      } else if (a.splits > 1) {
        a.part_lse[part] = lse;
      } else if (a.lse) {
        a.lse[row] = lse;
      }
    }
  }
  if (kCluster) {   // the parts' blocks share out the rows
    tc::cluster_sync();
    for (int r = split + a.splits * warp; r < rows; r += a.splits * kTokenWarps) {
      const uint32_t stat = tc::smem_u32(all + 16 * C::OP + r);
      float pm = -INFINITY, pl = 0.f;   // lane s: part s
      if (lane < a.splits) {
        uint32_t addr;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(stat), "r"(lane));
        pm = ld_cluster(addr);
        pl = ld_cluster(addr + 64);
      }
      float top = pm;
#pragma unroll
      for (int i = 4; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, i));
      top = __shfl_sync(kFull, top, 0);
      const float base = top == -INFINITY ? 0.f : top;
      const float f = lane < a.splits ? exp2f(pm - base) : 0.f;
      float total = f * pl;
#pragma unroll
      for (int i = 4; i; i >>= 1) total += __shfl_xor_sync(kFull, total, i);
      total = __shfl_sync(kFull, total, 0);
      const float inv = total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);
      float v[DC];
#pragma unroll
      for (int c = 0; c < DC; ++c) v[c] = 0.f;
      for (int s = 0; s < a.splits; ++s) {
        uint32_t addr;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(addr) : "r"(tc::smem_u32(all + r * C::OP + lane)), "r"(s));
        const float w = __shfl_sync(kFull, f, s);
#pragma unroll
        for (int c = 0; c < DC; ++c)
          if (32 * c + lane < a.dim) v[c] = fmaf(w, ld_cluster(addr + 128 * c), v[c]);
      }
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + row_offset(a, a.os, b, hk, r0 + r);
#pragma unroll
      for (int c = 0; c < DC; ++c)
        if (32 * c + lane < a.dim) dst[32 * c + lane] = __float2bfloat16_rn(v[c] * inv);
      if (a.lse && lane == 0)
        a.lse[((int64_t)b * a.kv_heads + hk) * a.rows + r0 + r] =
            total == 0.f ? -INFINITY : (base + log2f(total)) * kLn2;
    }
    tc::cluster_sync();   // no block leaves while its part is being read
  }
}

// delta of the backward pass where batch entries have few permitted keys, a block per 64
// packed query rows.  delta = sum_d dout out takes out as it was rounded to bf16; its
// error of up to 2^-8 |dout out| goes into every dS of the row, and where few keys share the
// row's weight that is not small beside dS = P (dP - delta) itself (one key: dS is 0, and
// the error all that remains).  With rows of v about zero, out and its error fall with the
// square root of the number of keys: for up to kExactKeys of them delta is taken here, as
// sum_j P_j dP_j from q, k, v, dout and lse (two products more); for more of them it stays as
// delta_kernel took it from out.  (A part that all rows of v have in common stays in out,
// while dq falls: with a mean as large as the spread, 64 channels, dq is off by 0.37% in norm
// at 256 keys, 0.9% at 4096 and 1.8% at 16384; 0.24% without it.  At every length it would be
// two products more beside the backward pass's seven.)
template <int DC>
__global__ void __launch_bounds__(128) delta_keys_kernel(const __grid_constant__ Args a) {
  using C = TokenCfg<DC>;
  __shared__ __align__(1024) uint8_t kt[32 * C::ROW];
  __shared__ __align__(1024) uint8_t vt[32 * C::ROW];
  __shared__ int permitted;
  if (threadIdx.x == 0) permitted = 0;
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int hk = blockIdx.y, b = blockIdx.z, r0 = blockIdx.x * 64 + 16 * warp;
  const int len = walk_end(a, b);
  const int64_t row0 = ((int64_t)b * a.kv_heads + hk) * a.rows;
  int count = len;
  if (a.key_mask && len > kExactKeys) {
    count = 0;   // no further than the answer needs
    for (int key0 = 0; key0 < len && count <= kExactKeys; key0 += 512) {
      int mine = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) mine += key_ok(a, b, len, key0 + 128 * i + threadIdx.x);
      mine = __reduce_add_sync(kFull, mine);
      __syncthreads();
      if (lane == 0) atomicAdd(&permitted, mine);
      __syncthreads();
      count = permitted;
    }
  }
  if (count > kExactKeys) return;   // delta_kernel's will do
  const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(a.k) + b * a.ks[0] + hk * a.ks[2];
  const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(a.v) + b * a.vs[0] + hk * a.vs[2];
  uint32_t qr[2 * DC][4], gr[2 * DC][4];   // rows g and g + 8 of q and dout, as A fragments
  float lse2[2], sum[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + 8 * i + g;
    const bool in = r < a.rows;
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) + (in ? row_offset(a, a.qs, b, hk, r) : 0);
    const __nv_bfloat16* gp = static_cast<const __nv_bfloat16*>(a.dout) + (in ? row_offset(a, a.dos, b, hk, r) : 0);
    lse2[i] = in ? a.lse_in[row0 + r] * kLog2e : INFINITY;
#pragma unroll
    for (int kk = 0; kk < 2 * DC; ++kk)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int d = 16 * kk + 8 * e + 2 * t;
        const bool real = in && d < a.dim;
        qr[kk][2 * e + i] = real ? *reinterpret_cast<const uint32_t*>(qp + d) : 0u;
        gr[kk][2 * e + i] = real ? *reinterpret_cast<const uint32_t*>(gp + d) : 0u;
      }
  }
  const float c2 = a.scale * kLog2e;
  for (int key0 = 0; key0 < len; key0 += 32) {
    const uint32_t w = __ballot_sync(kFull, key_ok(a, b, len, key0 + lane));
    if (w == 0) continue;   // the same in every warp
    __syncthreads();
    for (int e = threadIdx.x; e < 32 * C::CH; e += 128) {
      const int row = e / C::CH, c = e % C::CH;
      const bool real = (w >> row & 1u) && 8 * c < a.dim;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(kt + C::at(row, c)) =
          real ? *reinterpret_cast<const uint4*>(kp + (key0 + row) * a.ks[1] + 8 * c) : zero;
      *reinterpret_cast<uint4*>(vt + C::at(row, c)) =
          real ? *reinterpret_cast<const uint4*>(vp + (key0 + row) * a.vs[1] + 8 * c) : zero;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float s[2][4] = {}, dp[2][4] = {};
#pragma unroll
      for (int kk = 0; kk < 2 * DC; ++kk) {
        const uint32_t at = C::at(16 * h + (lane / 16) * 8 + lane % 8, 2 * kk + lane / 8 % 2);
        uint32_t f[4];
        ldm4(tc::smem_u32(kt) + at, f);
        mma16816(s[0], qr[kk][0], qr[kk][1], qr[kk][2], qr[kk][3], f[0], f[1]);
        mma16816(s[1], qr[kk][0], qr[kk][1], qr[kk][2], qr[kk][3], f[2], f[3]);
        ldm4(tc::smem_u32(vt) + at, f);
        mma16816(dp[0], gr[kk][0], gr[kk][1], gr[kk][2], gr[kk][3], f[0], f[1]);
        mma16816(dp[1], gr[kk][0], gr[kk][1], gr[kk][2], gr[kk][3], f[2], f[3]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (w >> (16 * h + 8 * i + 2 * t + e % 2) & 1u)
            sum[e / 2] = fmaf(exp2f(fmaf(s[i][e], c2, -lse2[e / 2])), dp[i][e], sum[e / 2]);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float d = quad_sum(sum[i]);
    const int r = r0 + 8 * i + g;
    if (t == 0 && r < a.rows) a.delta[row0 + r] = d;
  }
}

template <int DC, bool kCluster>
kfac_status launch_token(const Args& a, cudaStream_t st) {
  using C = TokenCfg<DC>;
  static OncePerDevice once;
  const kfac_status e = allow_smem(once, token_kernel<DC, kCluster>, C::SMEM);
  if (e != KFAC_OK) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(cdiv(a.rows, 16) * a.splits), a.kv_heads, a.batch);
  cfg.blockDim = dim3(kTokenWarps * 32);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = a.splits;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = kCluster ? 2 : 1;
  cudaLaunchKernelEx(&cfg, token_kernel<DC, kCluster>, a);
  count_launch();
  return check_launch();
}
template <int DC>
kfac_status dispatch_token(const Args& a, cudaStream_t st) {
  return a.splits > 1 && a.splits <= kTokenCluster ? launch_token<DC, true>(a, st)
                                                   : launch_token<DC, false>(a, st);
}

template <int DC>
kfac_status launch_delta_keys(const Args& a, cudaStream_t st) {
  launch_pdl(delta_keys_kernel<DC>, dim3((unsigned)cdiv(a.rows, 64), a.kv_heads, a.batch), dim3(128), 0, st, a);
  count_launch();
  return check_launch();
}

}  // namespace

kfac_status delta_keys(const Args& a, cudaStream_t st) {
  if (a.dim <= 32) return launch_delta_keys<1>(a, st);
  if (a.dim <= 64) return launch_delta_keys<2>(a, st);
  if (a.dim <= 96) return launch_delta_keys<3>(a, st);
  return launch_delta_keys<4>(a, st);
}

kfac_status token_forward(const Args& a, cudaStream_t st) {
  if (a.dim <= 32) return dispatch_token<1>(a, st);
  if (a.dim <= 64) return dispatch_token<2>(a, st);
  if (a.dim <= 96) return dispatch_token<3>(a, st);
  return dispatch_token<4>(a, st);
}

}  // namespace attn
}  // namespace kfac
