// Cross attention on the tensor cores (bf16): forward, and the backward pass.
//
// All three kernels are warp-specialised, one block per SM:
//   warp 0      TMA producer: tiles of 128 rows x 64-channel chunks, 128-byte swizzle
//   warp 1      MMA issuer (tcgen05, accumulators in TMEM)
//   warp 2      row statistics into shared memory (dK/dV role)
//   warps 4-11  two groups of 128 threads, one TMEM lane (score row) per thread
// Scores never leave the SM: S is read from TMEM into registers, P (or dS) goes back
// over it as bf16 and is the A operand of the next product straight from TMEM.
//
// Every wait is bounded (tc::mbar_wait); a role that gives up raises the block's abort
// flag, records KFAC_ERR_TIMEOUT in the operators' status word, and the block leaves
// NaN in its outputs.
#include "attn.cuh"
#include "tc_prims.cuh"
#include "tensor_map.cuh"

#include <algorithm>

namespace kfac {
namespace attn {

__device__ DevStatus g_op_status;

namespace {

constexpr int kTcThreads = 384;
constexpr int BT = 128;                    // rows of every tile
constexpr int kChunk = BT * 128;           // bytes of a 128-row, 64-channel chunk
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kNaN = __builtin_nanf("");

// What a block needs besides Args: how a coordinate of each tensor's map is formed
// (0: the axis is broadcast or has one entry).
struct MapMul {
  int head, batch;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&p);
}

// Bit i of w[c]: key key0 + 32 c + i is permitted.  Called by whole warps.
__device__ __forceinline__ void key_words(const Args& a, int b, int len, int key0,
                                          uint32_t (&w)[4]) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int n = len - (key0 + 32 * c);
    w[c] = n >= 32 ? kFull : n <= 0 ? 0u : (1u << n) - 1u;
    if (a.key_mask) w[c] &= __ballot_sync(kFull, key_ok(a, b, len, key0 + 32 * c + lane));
  }
}
__device__ __forceinline__ bool all_ok(const uint32_t (&w)[4]) {
  return (w[0] & w[1] & w[2] & w[3]) == kFull;
}

// Rows of a [128 x 64 NC] tile whose key is not permitted become zero: 0 x Inf or NaN
// in a product over keys would reach every row.  One warp; visible to the tensor
// cores afterwards.
template <int NC>
__device__ __forceinline__ void zero_rows(uint8_t* tile, const uint32_t (&w)[4]) {
  const int lane = threadIdx.x % 32;
  // lane = 16-byte column (8 per chunk row) x 4 rows at a time
#pragma unroll 1
  for (int r = lane / 8; r < BT; r += 4) {
    if (w[r / 32] >> (r % 32) & 1u) continue;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      *reinterpret_cast<uint4*>(tile + c * kChunk + r * 128 + (lane % 8) * 16) = make_uint4(0, 0, 0, 0);
  }
  tc::fence_proxy_async();
  __syncwarp();
}

template <int NC>
__device__ __forceinline__ void load_chunks(uint8_t* dst, const CUtensorMap* m, uint64_t* bar,
                                            int row, int head, int batch) {
  tc::mbar_expect_tx(bar, NC * kChunk);
#pragma unroll
  for (int c = 0; c < NC; ++c) tc::tma_load_4d(dst + c * kChunk, m, bar, 64 * c, row, head, batch);
}

// D[128 x 128] = A[128 x dim] . B[128 x dim]^T, both tiles in shared memory, channels
// contiguous.
__device__ __forceinline__ void mma_scores(uint32_t d, const uint8_t* a, const uint8_t* b,
                                           int ksteps) {
  constexpr uint32_t idesc = tc::make_idesc(1, 128, 128);
  const uint32_t sa = tc::smem_u32(a), sb = tc::smem_u32(b);
#pragma unroll 1
  for (int kk = 0; kk < ksteps; ++kk) {
    const uint32_t off = (uint32_t)(kk / 4 * kChunk + kk % 4 * 32);
    tc::umma_f16(d, tc::sdesc_kmajor_sw128(sa + off), tc::sdesc_kmajor_sw128(sb + off), idesc,
                 kk > 0);
  }
}
// D[128 x n] (+)= A[128 x 128] (TMEM, bf16; its second 64 columns of k start `half`
// TMEM columns after the first) . B, B the [128 x n] tile (rows = k).
__device__ __forceinline__ void mma_values(uint32_t d, uint32_t a, uint32_t half, const uint8_t* b,
                                           uint32_t idesc, bool accumulate) {
  const uint32_t sb = tc::smem_u32(b);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    tc::umma_f16_ts(d, a + (kk < 4 ? 0u : half) + (uint32_t)(kk % 4) * 8,
                    tc::sdesc_mnmajor_sw128(sb + kk * 2048, kChunk), idesc, accumulate || kk > 0);
}

// ------------------------------------------------------------------------- forward
//
// A block takes two tiles of 128 queries of one head against the keys of its part:
//   S_t = Q_t K^T          128 x 128 x dim, TMEM columns [128 t, 128 t + 128)
//   P_t = exp(S_t - m_t)   one thread per row: no shuffles for the maximum or the sum
//   O_t += P_t V           128 x dim x 128, TMEM columns [256 + 64 NC t, ...)
// Two tiles so that one's exponentials run under the other's products.  m_t is the
// row's reference maximum: it moves (and O_t, l_t are rescaled) only when the true
// maximum has grown past it by more than 2^8, which changes no result (P <= 2^8 fits
// bf16 as well as P <= 1) and leaves the rescaling out of almost every tile.
template <int NC> struct FwdCfg {
  static constexpr int TILE = NC * kChunk;
  static constexpr int STAGES = NC == 1 ? 3 : 2;
  static constexpr size_t SMEM = 1024 + (size_t)(2 + 2 * STAGES) * TILE + 256;
};
constexpr float kGrow = 8.f;

template <int NC>
__global__ void __launch_bounds__(kTcThreads, 1)
tc_forward_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap mq,
                  const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                  const MapMul xq, const MapMul xk, const MapMul xv) {
  using C = FwdCfg<NC>;
  constexpr int ST = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* Qs = smem;
  uint8_t* Ks = Qs + 2 * C::TILE;
  uint8_t* Vs = Ks + ST * C::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(Vs + ST * C::TILE);
  uint64_t *q_full = bars, *k_full = q_full + 2, *k_empty = k_full + ST, *v_full = k_empty + ST,
           *v_empty = v_full + ST, *s_full = v_empty + ST, *p_ready = s_full + 2,
           *o_full = p_ready + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_full + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(&q_full[t], 1);
      tc::mbar_init(&s_full[t], 1);
      tc::mbar_init(&p_ready[t], 4);
      tc::mbar_init(&o_full[t], 1);
    }
    for (int s = 0; s < ST; ++s) {
      tc::mbar_init(&k_full[s], 1);
      tc::mbar_init(&k_empty[s], 1);
      tc::mbar_init(&v_full[s], 1);
      tc::mbar_init(&v_empty[s], 1);
    }
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  const int split = (int)(blockIdx.x % a.splits);
  const int q0 = (int)(blockIdx.x / a.splits) * 2 * BT, h = blockIdx.y, b = blockIdx.z;
  const int hk = h / a.group;
  const int nt = q0 + BT < a.len_q ? 2 : 1;
  const int len = key_count(a, b);
  const int tiles = (len + BT - 1) / BT;
  const int t0 = (int)((int64_t)tiles * split / a.splits);
  const int n = (int)((int64_t)tiles * (split + 1) / a.splits) - t0;
  const int ksteps = (a.dim + 15) / 16;
  auto give_up = [&](int info) {
    *abort_flag = 1;
    if (lane == 0) report_error(&g_op_status, KFAC_ERR_TIMEOUT, -1, info);
  };

  if (warp == 0) {
    if (lane == 0 && n > 0) {  // -------------------------------------- TMA producer
      tc::tma_prefetch_desc(&mq);
      tc::tma_prefetch_desc(&mk);
      tc::tma_prefetch_desc(&mv);
      load_chunks<NC>(Qs, &mq, &q_full[0], q0, h * xq.head, b * xq.batch);
      int j = 0;
      for (; j < n; ++j) {
        const int s = j % ST;
        const uint32_t ph = (uint32_t)(j / ST) & 1u;
        if (!tc::mbar_wait(&k_empty[s], ph ^ 1, abort_flag)) break;
        load_chunks<NC>(Ks + s * C::TILE, &mk, &k_full[s], (t0 + j) * BT, hk * xk.head, b * xk.batch);
        if (j == 0 && nt == 2)
          load_chunks<NC>(Qs + C::TILE, &mq, &q_full[1], q0 + BT, h * xq.head, b * xq.batch);
        if (!tc::mbar_wait(&v_empty[s], ph ^ 1, abort_flag)) break;
        load_chunks<NC>(Vs + s * C::TILE, &mv, &v_full[s], (t0 + j) * BT, hk * xv.head, b * xv.batch);
      }
      if (j < n) {   // winding down: let the copies in flight land before the block ends
        give_up(101);
        int never = 0;
        for (int s = 0; s < ST; ++s) {
          tc::mbar_wait(&k_full[s], (uint32_t)(j / ST) & 1u, &never, 1 << 20);
          tc::mbar_wait(&v_full[s], (uint32_t)(j / ST) & 1u, &never, 1 << 20);
        }
      }
    }
  } else if (warp == 1) {  // ------------------------------------------- MMA issuer
    const uint32_t idesc_o = tc::make_idesc(1, 128, ksteps * 16) | tc::kIdescMnB;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool ok = __all_sync(kFull, tc::mbar_wait(bar, parity, abort_flag));
      if (!ok) give_up(102);
      tc::tc_fence_after();
      return ok;
    };
    bool ok = n > 0 && wait(&k_full[0], 0);
    for (int t = 0; t < nt && ok; ++t) {
      ok = wait(&q_full[t], 0);
      if (ok && lane == 0) {
        mma_scores(tmem + 128 * t, Qs + t * C::TILE, Ks, ksteps);
        tc::umma_commit(&s_full[t]);
        if (t == nt - 1) tc::umma_commit(&k_empty[0]);
      }
    }
    for (int j = 0; j < n && ok; ++j) {
      const int s = j % ST, s1 = (j + 1) % ST;
      for (int t = 0; t < nt && ok; ++t) {
        if (t == 0) {
          ok = wait(&v_full[s], (uint32_t)(j / ST) & 1u);
          uint32_t w[4];
          key_words(a, b, len, (t0 + j) * BT, w);
          if (ok && !all_ok(w)) zero_rows<NC>(Vs + s * C::TILE, w);
        }
        ok = ok && wait(&p_ready[t], (uint32_t)j & 1u);
        if (ok && lane == 0) {
          mma_values(tmem + 256 + 64 * NC * t, tmem + 128 * t, 32, Vs + s * C::TILE, idesc_o, j > 0);
          if (t == nt - 1) tc::umma_commit(&v_empty[s]);
          if (j == n - 1) tc::umma_commit(&o_full[t]);
        }
        if (j + 1 < n && ok) {
          if (t == 0) ok = wait(&k_full[s1], (uint32_t)((j + 1) / ST) & 1u);
          if (ok && lane == 0) {
            mma_scores(tmem + 128 * t, Qs + t * C::TILE, Ks + s1 * C::TILE, ksteps);
            tc::umma_commit(&s_full[t]);
            if (t == nt - 1) tc::umma_commit(&k_empty[s1]);
          }
        }
        __syncwarp();
      }
    }
  } else if (warp >= 4 && (warp - 4) / 4 < nt) {  // -------------- softmax, epilogue
    const int t = (warp - 4) / 4;
    const uint32_t lanes = (uint32_t)(warp % 4) * 32 << 16;
    const uint32_t ts = tmem + 128 * t + lanes, to = tmem + 256 + 64 * NC * t + lanes;
    const float c2 = a.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n && ok; ++j) {
      uint32_t w[4];
      key_words(a, b, len, (t0 + j) * BT, w);
      ok = __all_sync(kFull, tc::mbar_wait(&s_full[t], (uint32_t)j & 1u, abort_flag));
      if (!ok) break;
      tc::tc_fence_after();
      uint32_t r[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::tmem_ld32_issue(ts + 32 * c, r[c]);
      tc::tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::tmem_ld_use(r[c]);
      if (!all_ok(w)) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(w[c] >> i & 1u)) r[c][i] = 0xff800000u;   // -infinity
      }
      float top[4] = {m, m, m, m};
#pragma unroll
      for (int i = 0; i < 32; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) top[c] = fmaxf(top[c], __uint_as_float(r[c][i]));
      const float grown = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      if (j == 0) {
        m = grown;
      } else if (__any_sync(kFull, (grown - m) * c2 > kGrow)) {
        const float f = grown == m ? 1.f : ex2((m - grown) * c2);
        m = grown;
        l *= f;
        for (int c = 0; c < ksteps * 16; c += 32) {
          uint32_t o[32];
          tc::tmem_ld32_issue(to + c, o);
          tc::tmem_ld_wait();
          tc::tmem_ld_use(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          tc::tmem_st32(to + c, o);
        }
      }
      const float base = m == -INFINITY ? 0.f : m * c2;   // nothing permitted so far
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t p[32];
#pragma unroll
        for (int cc = 0; cc < 2; ++cc)
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const int c = 2 * half + cc;
            const float x = ex2(fmaf(__uint_as_float(r[c][i]), c2, -base));
            const float y = ex2(fmaf(__uint_as_float(r[c][i + 1]), c2, -base));
            sum[i % 4] += x;
            sum[i % 4 + 1] += y;
            p[16 * cc + i / 2] = pack_bf16(x, y);
          }
        tc::tmem_st32(ts + 32 * half, p);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tc::tmem_st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&p_ready[t]);
    }
    if (n > 0 && ok) ok = __all_sync(kFull, tc::mbar_wait(&o_full[t], 0, abort_flag));
    if (!ok) give_up(103);
    tc::tc_fence_after();
    const int q = q0 + BT * t + 32 * (warp % 4) + lane;
    const float inv = !ok ? kNaN : l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    const float lse = !ok ? kNaN : l == 0.f ? -INFINITY : (m * c2 + log2f(l)) * kLn2;
    const int64_t row = ((int64_t)b * a.heads + h) * a.len_q + q;   // of the statistics
    const int64_t part = (int64_t)split * a.batch * a.heads * a.len_q + row;
    for (int c = 0; c < a.dim; c += 32) {
      uint32_t o[32];
      if (n > 0) {
        tc::tmem_ld32_issue(to + c, o);
        tc::tmem_ld_wait();
        tc::tmem_ld_use(o);
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = n > 0 ? __float_as_uint(__uint_as_float(o[i]) * inv) : 0u;
      if (q < a.len_q) {
        if (a.splits == 1) {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + b * a.os[0] + q * a.os[1] + h * a.os[2];
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            if (c + i < a.dim) {
              uint4 u;
              u.x = pack_bf16(__uint_as_float(o[i]), __uint_as_float(o[i + 1]));
              u.y = pack_bf16(__uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
              u.z = pack_bf16(__uint_as_float(o[i + 4]), __uint_as_float(o[i + 5]));
              u.w = pack_bf16(__uint_as_float(o[i + 6]), __uint_as_float(o[i + 7]));
              *reinterpret_cast<uint4*>(dst + c + i) = u;
            }
        } else {
          float* dst = a.part_o + part * a.dim;
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            if (c + i < a.dim)
              *reinterpret_cast<uint4*>(dst + c + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
      }
    }
    if (q < a.len_q) {
      if (a.splits > 1) a.part_lse[part] = lse;
      else if (a.lse) a.lse[row] = lse;
    }
    tc::tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------------ tensor maps

// [batch, rows, heads, dim] as a 4-D map (channels, rows, heads, batch), boxes of 128
// rows x 64 channels; what lies past dim or rows reads as zero.  An axis of stride 0
// or of one entry has one entry in the map and coordinate 0.
bool make_map(CUtensorMap* m, MapMul* mul, const void* p, const int64_t* s, int dim, int rows,
              int heads, int batch) {
  auto fn = encode_fn();
  if (!fn) return false;
  mul->head = heads > 1 && s[2] != 0;
  mul->batch = batch > 1 && s[0] != 0;
  cuuint64_t dims[4] = {(cuuint64_t)dim, (cuuint64_t)rows, mul->head ? (cuuint64_t)heads : 1u,
                        mul->batch ? (cuuint64_t)batch : 1u};
  cuuint64_t st[3] = {rows > 1 ? (cuuint64_t)s[1] * 2 : 16u, mul->head ? (cuuint64_t)s[2] * 2 : 16u,
                      mul->batch ? (cuuint64_t)s[0] * 2 : 16u};
  cuuint32_t box[4] = {64u, (cuuint32_t)BT, 1u, 1u}, es[4] = {1u, 1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p), dims, st, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows that TMA can address and 16-byte vectors can read and write.
bool rows_ok(const void* p, const int64_t* s, int rows, int heads, int batch) {
  const int64_t n[3] = {batch, rows, heads};
  if ((uintptr_t)p % 16) return false;
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (s[i] % 8 || s[i] >= (int64_t(1) << 38))) return false;
  return rows <= 1 || s[1] > 0;
}

template <int NC>
kfac_status launch_tc_forward(const Args& a, cudaStream_t st) {
  using C = FwdCfg<NC>;
  static const bool ok = cudaFuncSetAttribute(tc_forward_kernel<NC>,
                                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              (int)C::SMEM) == cudaSuccess;
  CUtensorMap mq, mk, mv;
  MapMul xq, xk, xv;
  if (!ok || !make_map(&mq, &xq, a.q, a.qs, a.dim, a.len_q, a.heads, a.batch) ||
      !make_map(&mk, &xk, a.k, a.ks, a.dim, a.len_kv, a.kv_heads, a.batch) ||
      !make_map(&mv, &xv, a.v, a.vs, a.dim, a.len_kv, a.kv_heads, a.batch))
    return KFAC_ERR_CUDA;
  const dim3 grid((unsigned)(cdiv(a.len_q, 2 * BT) * a.splits), a.heads, a.batch);
  launch_pdl(tc_forward_kernel<NC>, grid, dim3(kTcThreads), C::SMEM, st, a, mq, mk, mv, xq, xk, xv);
  count_launch();
  return check_launch();
}

}  // namespace

bool tc_forward_ok(const Args& a) {
  return a.dim % 8 == 0 && a.len_kv > 0 && rows_ok(a.q, a.qs, a.len_q, a.heads, a.batch) &&
         rows_ok(a.k, a.ks, a.len_kv, a.kv_heads, a.batch) &&
         rows_ok(a.v, a.vs, a.len_kv, a.kv_heads, a.batch) &&
         rows_ok(a.out, a.os, a.len_q, a.heads, a.batch);
}

kfac_status tc_forward(const Args& a, cudaStream_t st) {
  return a.dim <= 64 ? launch_tc_forward<1>(a, st) : launch_tc_forward<2>(a, st);
}

}  // namespace attn
}  // namespace kfac

using namespace kfac;

extern "C" kfac_status kfac_operator_status(int* info) {
  if (cudaDeviceSynchronize() != cudaSuccess) return KFAC_ERR_CUDA;
  DevStatus s{}, zero{};
  if (cudaMemcpyFromSymbol(&s, attn::g_op_status, sizeof(s)) != cudaSuccess) return KFAC_ERR_CUDA;
  if (info) *info = s.code ? s.info : 0;
  if (s.code && cudaMemcpyToSymbol(attn::g_op_status, &zero, sizeof(zero)) != cudaSuccess)
    return KFAC_ERR_CUDA;
  return (kfac_status)s.code;
}
