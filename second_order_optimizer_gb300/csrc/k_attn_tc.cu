// Cross attention on the tensor cores (bf16): forward, and the backward pass.
//
// Warp-specialised blocks:
//   warp 0    TMA producer: tiles of 128 rows x 64-channel chunks, 128-byte swizzle
//   warp 1    MMA issuer (tcgen05, accumulators in TMEM), converged, one elected lane issuing
//   warp 2    key masks and the rows they clear; row statistics of the dK/dV blocks
//   warps 4-  groups of four: one TMEM lane (score row) per thread
// Scores never leave the SM: S is read from TMEM into registers, P (or dS) goes back
// over it as bf16 and is the A operand of the next product straight from TMEM.
//
// Every wait is bounded (tc::mbar_wait); a role that gives up raises the block's abort
// flag, records KFAC_ERR_TIMEOUT in the operators' status word, and the block leaves
// NaN in its outputs.  Such a block does not let its shared and tensor memory go before the
// producer's copies have landed and the issuer's products have ended (bounded as well).
#include "attn.cuh"
#include "ring.h"
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two fp32 operations in one instruction, on pairs of registers.
struct F2 { uint64_t v; };
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ F2 f2(uint32_t x, uint32_t y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ void unpack(F2 a, float* x, float* y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*x), "=f"(*y) : "l"(a.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&p);
}

// Bit i of w[c]: key key0 + 32 c + i is below len.
__device__ __forceinline__ void len_words(int len, int key0, uint32_t (&w)[4]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int n = len - (key0 + 32 * c);
    w[c] = n >= 32 ? kFull : n <= 0 ? 0u : (1u << n) - 1u;
  }
}
__device__ __forceinline__ bool all_ok(const uint32_t (&w)[4]) {
  return (w[0] & w[1] & w[2] & w[3]) == kFull;
}

// Rows of a [128 x 64 NC] tile whose key is not permitted become zero: 0 x Inf or NaN
// in a product over keys would reach every row.  One warp, one row per lane (starting
// at different 16-byte columns: no bank is written twice at once); visible to the
// tensor cores afterwards.
template <int NC>
__device__ __forceinline__ void zero_rows(uint8_t* tile, const uint32_t (&w)[4]) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!(w[i] >> lane & 1u)) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<uint4*>(tile + c * kChunk + (32 * i + lane) * 128 + (k + lane) % 8 * 16) =
              make_uint4(0, 0, 0, 0);
    }
  tc::fence_proxy_async();
  __syncwarp();
}

// The same warp's walk over a block's key tiles: the words of tile `key0` (the mask's
// bytes of the next tile are already on their way), published to the score warps.
struct MaskWalk {
  uint8_t next[4];
  __device__ __forceinline__ void fetch(const Args& a, int b, int len, int key0) {
    if (!a.key_mask) return;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int key = key0 + 32 * c + (int)(threadIdx.x % 32);
      next[c] = key < len ? __ldg(a.key_mask + (int64_t)b * a.len_kv + key) : (uint8_t)0;
    }
  }
  __device__ __forceinline__ void words(const Args& a, int len, int key0, uint32_t (&w)[4]) const {
    len_words(len, key0, w);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (a.key_mask) w[c] &= __ballot_sync(kFull, next[c] != 0);
    }
  }
};
template <int NC>
__device__ __forceinline__ void load_chunks(uint8_t* dst, const CUtensorMap* m, uint64_t* bar,
                                            int row, int head, int batch) {
  tc::mbar_expect_tx(bar, NC * kChunk);
#pragma unroll
  for (int c = 0; c < NC; ++c) tc::tma_load_4d(dst + c * kChunk, m, bar, 64 * c, row, head, batch);
}

constexpr long long kLandCycles = 1 << 20;   // 0.5 ms
// The copies behind a barrier that was used this often, or behind a ring's.
__device__ __forceinline__ void land(uint64_t* bar, int uses) {
  int never = 0;
  if (uses > 0) tc::mbar_wait(bar, ring_last_parity(uses), &never, kLandCycles);
}
template <int kStages> __device__ __forceinline__ void land_ring(uint64_t* bars, int issued) {
  for (int s = 0; s < kStages; ++s) land(&bars[s], ring_uses(issued, s, kStages));
}
// Everything that this warp has issued.  `bar` is used for nothing else.
__device__ __forceinline__ void end_mmas(uint64_t* bar) {
  int never = 0;
  tc::umma_commit_by(tc::elect_leader(), bar);
  tc::mbar_wait(bar, 0, &never, kLandCycles);
}

// D[128 x 128] = A[128 x dim] . B[128 x dim]^T, both tiles in shared memory, channels
// contiguous.
__device__ __forceinline__ void mma_scores(uint32_t leader, uint32_t d, const uint8_t* a, const uint8_t* b,
                                           int ksteps) {
  constexpr uint32_t idesc = tc::make_idesc(1, 128, 128);
  const uint64_t da = tc::sdesc_kmajor_sw128(tc::smem_u32(a)), db = tc::sdesc_kmajor_sw128(tc::smem_u32(b));
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {   // addresses in the descriptors count 16 bytes
    const uint64_t off = (uint64_t)((kk / 4 * kChunk + kk % 4 * 32) >> 4);
    if (kk < ksteps) tc::umma_f16_by(leader, d, da + off, db + off, idesc, kk > 0);
  }
}
// D[128 x n] (+)= A[128 x 64] (TMEM, bf16) . B, 64 rows (k) of n channels in shared
// memory.
__device__ __forceinline__ void mma_values(uint32_t leader, uint32_t d, uint32_t a, const uint8_t* b,
                                           uint32_t idesc, bool accumulate) {
  const uint64_t db = tc::sdesc_mnmajor_sw128(tc::smem_u32(b), kChunk);
#pragma unroll
  for (int kk = 0; kk < 4; ++kk)   // 16 k: two groups of eight 128-byte rows
    tc::umma_f16_ts_by(leader, d, a + (uint32_t)kk * 8, db + (kk * 2048 >> 4), idesc,
                       accumulate || kk > 0);
}
constexpr int kHalf = 64 * 128;   // bytes from a tile's row 0 to its row 64

// ------------------------------------------------------------------------- forward
//
// A block takes NT tiles of 128 queries of one head against the keys of its part:
//   S_t = Q_t K^T          128 x 128 x dim, TMEM columns [128 t, 128 t + 128)
//   P_t = exp(S_t - m_t)   one thread per row: no shuffles for the maximum or the sum
//   O_t += P_t V           128 x dim x 128, TMEM columns [128 NT + 64 NC t, ...)
// Two tiles (or two blocks of one) per SM, so that one's exponentials run under the
// other's products.  The chain of a tile - S, exponentials, P V, S - is what bounds the
// kernel, so it is kept short: P is handed over in halves of 64 keys, and a half's
// exponentials do not wait for its maximum.  They are taken against the row's reference
// maximum m_t so far; only when the half's own maximum, found alongside, has grown past it
// by more than 2^8 are they taken again and O_t, l_t rescaled (in a tile's second half the
// products of the first must end before).  A reference that lags changes P, l and O by a
// power of two at most: P <= 2^8, and O overflows only where 2^8 len_kv |v| does.  (The second
// half may not wait longer for it: at 2^90 a row that grows by 60 within a tile took |v| past
// 2.7e11 to infinity.)
// Measured on 8 x 2048 queries, 4096 keys (ragged: 56 % of them permitted), 16 heads x 128:
// 222 us, 1390 TFLOP/s, the tensor pipe active in 66 % of the cycles.  What was tried and cost
// more: S in two buffers of 64 keys (a quarter more: twice the hand-overs), two groups of warps
// per tile (a twentieth).
template <int NC, int NT> struct FwdCfg {
  static constexpr int TILE = NC * kChunk;
  static constexpr int THREADS = 128 + 128 * NT;
  static constexpr int STAGES = (NC == 1 ? 3 : 2) - (NT == 1 ? 1 : 0);
  static constexpr int TMEM = 256 * NT, OCOL = 128 * NT;   // columns, and where O starts
  static constexpr size_t SMEM = (size_t)(NT + 2 * STAGES) * TILE + 512;
};
constexpr float kGrow = 8.f;

template <int NC, int NT>
__global__ void __launch_bounds__(FwdCfg<NC, NT>::THREADS, 3 - NT)
tc_forward_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap mq,
                  const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                  const MapMul xq, const MapMul xk, const MapMul xv) {
  using C = FwdCfg<NC, NT>;
  constexpr int ST = C::STAGES;
  extern __shared__ __align__(1024) uint8_t smem[];   // the 128-byte swizzle's period
  uint8_t* Qs = smem;
  uint8_t* Ks = Qs + NT * C::TILE;
  uint8_t* Vs = Ks + ST * C::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(Vs + ST * C::TILE);
  uint64_t *q_full = bars, *k_full = q_full + 2, *k_empty = k_full + ST, *v_full = k_empty + ST,
           *v_empty = v_full + ST, *v_ready = v_empty + ST, *w_full = v_ready + ST,
           *s_full = w_full + ST, *p_ready = s_full + 2 /* [2 t + half] */, *half_done = p_ready + 4,
           *o_full = half_done + 2, *ended = o_full + 2 /* and one that keeps `words` aligned */;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ended + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint4* words = reinterpret_cast<uint4*>(tmem_slot + 4);   // [ST] permitted keys of a tile
  const int warp = __shfl_sync(kFull, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(&q_full[t], 1);
      tc::mbar_init(&s_full[t], 1);
      tc::mbar_init(&p_ready[2 * t], 4);
      tc::mbar_init(&p_ready[2 * t + 1], 4);
      tc::mbar_init(&half_done[t], 1);
      tc::mbar_init(&o_full[t], 1);
    }
    tc::mbar_init(ended, 1);
    for (int s = 0; s < ST; ++s) {
      tc::mbar_init(&k_full[s], 1);
      tc::mbar_init(&k_empty[s], 1);
      tc::mbar_init(&v_full[s], 1);
      tc::mbar_init(&v_empty[s], 1);
      tc::mbar_init(&v_ready[s], 1);
      tc::mbar_init(&w_full[s], 1);
    }
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, C::TMEM);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, *tmem_slot, 0);
  pdl_wait();
  pdl_trigger();

  const int split = (int)(blockIdx.x % a.splits);
  const int q0 = (int)(blockIdx.x / a.splits) * NT * BT, h = blockIdx.y, b = blockIdx.z;
  const int hk = h / a.group;
  const int nt = NT == 2 && q0 + BT < a.len_q ? 2 : 1;
  const int len = __shfl_sync(kFull, walk_end(a, b), 0);   // known to be warp-uniform
  const int tiles = (len + BT - 1) / BT;
  const int t0 = (int)((int64_t)tiles * split / a.splits);
  const int n = (int)((int64_t)tiles * (split + 1) / a.splits) - t0;
  const int ksteps = (a.dim + 15) / 16;
  int ks = 0, vs = 0;   // the producer's: tiles of k and v issued
  auto give_up = [&](int info) {
    *abort_flag = 1;
    if (lane == 0) report_error(&g_op_status, KFAC_ERR_TIMEOUT, -1, info);
  };

  if (warp < 4) {
  if (warp == 0) {
    if (lane == 0 && n > 0) {  // -------------------------------------- TMA producer
      tc::tma_prefetch_desc(&mq);
      tc::tma_prefetch_desc(&mk);
      tc::tma_prefetch_desc(&mv);
      load_chunks<NC>(Qs, &mq, &q_full[0], q0, h * xq.head, b * xq.batch);
      for (int j = 0; j < n; ++j) {
        const int s = j % ST;
        const uint32_t ph = (uint32_t)(j / ST) & 1u;
        if (!tc::mbar_wait(&k_empty[s], ph ^ 1, abort_flag)) break;
        load_chunks<NC>(Ks + s * C::TILE, &mk, &k_full[s], (t0 + j) * BT, hk * xk.head, b * xk.batch);
        ++ks;
        if (j == 0 && nt == 2)
          load_chunks<NC>(Qs + C::TILE, &mq, &q_full[1], q0 + BT, h * xq.head, b * xq.batch);
        if (!tc::mbar_wait(&v_empty[s], ph ^ 1, abort_flag)) break;
        load_chunks<NC>(Vs + s * C::TILE, &mv, &v_full[s], (t0 + j) * BT, hk * xv.head, b * xv.batch);
        ++vs;
      }
      if (vs < n) give_up(101);
    }
  } else if (warp == 1) {
    if (n > 0) {  // ----------------------------------------------------- MMA issuer
      const uint32_t leader = tc::elect_leader();
      const uint32_t idesc_o = tc::make_idesc(1, 128, ksteps * 16) | tc::kIdescMnB;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = __all_sync(kFull, tc::mbar_wait(bar, parity, abort_flag));
        if (!ok) give_up(102);
        return ok;
      };
      bool ok = wait(&k_full[0], 0);
      for (int t = 0; t < nt && ok; ++t) {
        if (!(ok = wait(&q_full[t], 0))) break;
        mma_scores(leader, tmem + 128 * t, Qs + t * C::TILE, Ks, ksteps);
        tc::umma_commit_by(leader, &s_full[t]);
        if (t == nt - 1) tc::umma_commit_by(leader, &k_empty[0]);
      }
      for (int j = 0; j < n && ok; ++j) {
        const int s = j % ST, s1 = (j + 1) % ST;
        if (!(ok = wait(&v_ready[s], (uint32_t)(j / ST) & 1u))) break;
        for (int t = 0; t < nt; ++t) {
          for (int half = 0; half < 2; ++half) {
            if (!(ok = wait(&p_ready[2 * t + half], (uint32_t)j & 1u))) break;
            tc::tc_fence_after();
            mma_values(leader, tmem + C::OCOL + 64 * NC * t, tmem + 128 * t + 32 * half,
                       Vs + s * C::TILE + half * kHalf, idesc_o, j > 0 || half > 0);
            if (half == 0) tc::umma_commit_by(leader, &half_done[t]);
          }
          if (!ok) break;
          if (t == nt - 1) tc::umma_commit_by(leader, &v_empty[s]);
          if (j == n - 1) tc::umma_commit_by(leader, &o_full[t]);
          if (j + 1 < n) {
            if (t == 0 && !(ok = wait(&k_full[s1], (uint32_t)((j + 1) / ST) & 1u))) break;
            mma_scores(leader, tmem + 128 * t, Qs + t * C::TILE, Ks + s1 * C::TILE, ksteps);
            tc::umma_commit_by(leader, &s_full[t]);
            if (t == nt - 1) tc::umma_commit_by(leader, &k_empty[s1]);
          }
        }
      }
    }
  } else if (warp == 2) {  // ------------------------------------------- key mask
    MaskWalk mask;
    mask.fetch(a, b, len, t0 * BT);
    for (int j = 0; j < n; ++j) {
      const int s = j % ST, key0 = (t0 + j) * BT;
      const uint32_t ph = (uint32_t)(j / ST) & 1u;
      uint32_t w[4];
      mask.words(a, len, key0, w);
      mask.fetch(a, b, len, key0 + BT);
      // the slot's last tile has been multiplied, so its words have been read
      bool ok = tc::mbar_wait(&v_empty[s], ph ^ 1, abort_flag);
      if (ok && lane == 0) {
        words[s] = make_uint4(w[0], w[1], w[2], w[3]);
        tc::mbar_arrive(&w_full[s]);
      }
      ok = __all_sync(kFull, ok && tc::mbar_wait(&v_full[s], ph, abort_flag));
      if (!ok) {
        give_up(104);
        break;
      }
      if (!all_ok(w)) zero_rows<NC>(Vs + s * C::TILE, w);
      if (lane == 0) tc::mbar_arrive(&v_ready[s]);
    }
  }
  } else {
  if ((warp - 4) / 4 < nt) {  // ---------------------------------- softmax, epilogue
    const int t = (warp - 4) / 4;
    const uint32_t lanes = (uint32_t)(warp % 4) * 32 << 16;
    const uint32_t ts = tmem + 128 * t + lanes, to = tmem + C::OCOL + 64 * NC * t + lanes;
    const float c2 = a.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n && ok; ++j) {
      ok = __all_sync(kFull, tc::mbar_wait(&s_full[t], (uint32_t)j & 1u, abort_flag) &&
                                 (!a.key_mask || tc::mbar_wait(&w_full[j % ST], (uint32_t)(j / ST) & 1u,
                                                               abort_flag)));
      if (!ok) break;
      tc::tc_fence_after();
      uint32_t w[4];
      if (a.key_mask) {
        const uint4 u = words[j % ST];
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
      } else {
        len_words(len, (t0 + j) * BT, w);
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t r[2][32];
        auto load = [&]() {
          tc::tmem_ld32_issue(ts + 64 * half, r[0]);
          tc::tmem_ld32_issue(ts + 64 * half + 32, r[1]);
          tc::tmem_ld_wait();
          tc::tmem_ld_use(r[0]);
          tc::tmem_ld_use(r[1]);
          if ((w[2 * half] & w[2 * half + 1]) != kFull) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(w[2 * half + c] >> e & 1u)) r[c][e] = 0xff800000u;   // -infinity
          }
        };
        uint32_t p[32];
        F2 sum[2];
        float top[4];
        auto exponentials = [&]() {
          const float base = m == -INFINITY ? 0.f : m * c2;   // nothing permitted so far
          const F2 cc2 = f2(c2, c2), nb2 = f2(-base, -base);
          sum[0] = sum[1] = f2(0.f, 0.f);
          top[0] = top[1] = top[2] = top[3] = m;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t u = r[e / 16][2 * e % 32], v = r[e / 16][2 * e % 32 + 1];
            float x, y;
            unpack(fma2(f2(u, v), cc2, nb2), &x, &y);
            top[e % 4] = max3(top[e % 4], __uint_as_float(u), __uint_as_float(v));
            x = ex2(x);
            y = ex2(y);
            sum[e % 2] = add2(sum[e % 2], f2(x, y));
            p[e] = pack_bf16(x, y);
          }
        };
        load();
        exponentials();
        const float grown = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        // (m = -infinity: any key counts as growth)
        if (__any_sync(kFull, (grown - m) * c2 > kGrow)) {
          if (half == 1) ok = __all_sync(kFull, tc::mbar_wait(&half_done[t], (uint32_t)j & 1u, abort_flag));
          if (!ok) break;
          tc::tc_fence_after();
          const float f = grown == m ? 1.f : ex2((m - grown) * c2);
          m = grown;
          l *= f;
          for (int c = 0; c < ksteps * 16 && j + half > 0; c += 32) {
            uint32_t o[32];
            tc::tmem_ld32_issue(to + c, o);
            tc::tmem_ld_wait();
            tc::tmem_ld_use(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tc::tmem_st32(to + c, o);
          }
          load();
          exponentials();
        }
        tc::tmem_st32(ts + 32 * half, p);
        float l0, l1;
        unpack(add2(sum[0], sum[1]), &l0, &l1);
        l += l0 + l1;
        tc::tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&p_ready[2 * t + half]);
      }
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
  }
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) {
      land(&q_full[0], n > 0);
      land(&q_full[1], nt == 2 && ks > 0);
      land_ring<ST>(k_full, ks);
      land_ring<ST>(v_full, vs);
    }
    if (warp == 1) end_mmas(ended);
    __syncthreads();
  }
  if (warp == 1) tc::tmem_dealloc(tmem, C::TMEM);
}

// ------------------------------------------------------------------------ backward
//
// One launch, two kinds of blocks, each recomputing S and dO V^T for its tiles: seven
// products in all instead of the five that one pass would take, but every output has
// one block that sums it in TMEM in a fixed order - no atomics, no fp32 dQ in memory,
// and the query heads that share a key head are summed where they are produced.
//
// dK/dV block: 128 keys, all query tiles of the group's heads.  One TMEM lane per key:
//   S^T = K Q^T, dP^T = V dO^T          (TMEM columns 0.., 128..)
//   P^T = exp(S^T - lse) over S^T;      dV += P^T dO    (columns 256..)
//   dS^T = P^T (dP^T - delta) over dP^T; dK += dS^T Q   (columns 256 + 64 NC..)
// The issuing order dP(i), dV(i), S(i+1), dK(i) lets P(i+1) run under dK(i) and
// dP(i+1), and dS(i) under dV(i) and S(i+1).
// With 64 channels, where the exponentials are the longer part, there is room for a second
// S: dP(i), S(i+1), dV(i), dK(i) - the score warps never wait for S.
//
// dQ block: 128 queries of one head, all tiles of permitted keys.  One lane per query:
//   S = Q K^T (columns 0..), dP = dO V^T (two buffers, 128.. and 256..)
//   dS = P (dP - delta) over dP; dQ += dS K (384..)
// Issuing order S(j+1), dP(j+1), dQ(j): S is free once it has been read, so both operands
// of dS(j+1) are there when dS(j) is done.  (With two buffers of S and one of dP, dP(j+1)
// waited for dQ(j): 2870 cycles a step; three products of 128 x 128 x 128 take 1536.)
//
// Two groups of four warps share a tile's columns, 64 each.
// Measured: 8 x 2048 queries, 4096 keys (56 % of them permitted), 16 heads x 128: 770 us, 1400
// TFLOP/s of the seven products, the tensor pipe active in 64 % of the cycles; 5 x 577, 1531, 16
// heads on 4 x 64: 69 us, 35 % (a block's set-up, chain and end are not hidden).
constexpr int kBwdBars = 26;   // then the TMEM slot and abort flag, then the mask words
template <int NC> struct BwdCfg {
  static constexpr int TILE = NC * kChunk;
  static constexpr int STATS = 2 * 2 * BT * 4;   // two stages of 128 lse and 128 delta
  static constexpr size_t SMEM = (size_t)7 * TILE + STATS + 512;
  static_assert(SMEM <= 227 * 1024, "shared memory of one block");
};

__device__ __forceinline__ void store_row(const uint32_t (&o)[32], __nv_bfloat16* dst, int c, int dim,
                                          float f, bool zero) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    if (c + i < dim) {
      uint32_t u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        u[k] = zero ? 0u : pack_bf16(__uint_as_float(o[i + 2 * k]) * f, __uint_as_float(o[i + 2 * k + 1]) * f);
      *reinterpret_cast<uint4*>(dst + c + i) = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// The same to a part's fp32 sums.
__device__ __forceinline__ void store_part(const uint32_t (&o)[32], float* dst, int c, int dim,
                                           bool ok, bool zero) {
#pragma unroll
  for (int i = 0; i < 32; i += 4)
    if (c + i < dim) {
      float4 v = make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]),
                             __uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
      if (zero) v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!ok) v = make_float4(kNaN, kNaN, kNaN, kNaN);
      *reinterpret_cast<float4*>(dst + c + i) = v;
    }
}

struct BwdMaps {
  CUtensorMap q, k, v, g;
  MapMul xq, xk, xv, xg;
};

template <int NC>
__device__ __forceinline__ void dkv_block(const Args& a, const BwdMaps& mp, int tile, int split, int hk, int b, uint8_t* smem,
                                          uint64_t* bars, volatile int* abort_flag, uint32_t tmem) {
  using C = BwdCfg<NC>;
  uint8_t *Ks = smem, *Vs = Ks + C::TILE, *Qs = Vs + C::TILE, *Gs = Qs + 3 * C::TILE;
  float* stats = reinterpret_cast<float*>(Gs + 2 * C::TILE);   // [2][lse 128, delta 128]
  uint64_t *kv_full = bars, *q_full = bars + 1, *q_empty = bars + 4, *g_full = bars + 7,
           *g_empty = bars + 9, *dp_full = bars + 12, *p_ready = bars + 13,
           *ds_ready = bars + 14, *st_full = bars + 15, *st_empty = bars + 17, *done = bars + 19,
           *kv_ready = bars + 20, *ended = bars + 22;
  // S^T of step i: one buffer, or with 64 channels two (the second behind dK)
  auto s_full = [&](int i) { return NC == 1 && i % 2 ? bars + 21 : bars + 11; };
  auto s_phase = [&](int i) { return (uint32_t)(NC == 1 ? i / 2 : i) & 1u; };
  auto s_at = [&](int i) { return tmem + (NC == 1 && i % 2 ? 384u : 0u); };
  const int warp = __shfl_sync(kFull, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int k0 = tile * BT;
  const int len = __shfl_sync(kFull, walk_end(a, b), 0);   // known to be warp-uniform
  const int qtiles = (a.len_q + BT - 1) / BT;
  // this part of the group's query tiles
  const int steps = k0 < len ? a.group * qtiles : 0;
  const int first = (int)((int64_t)steps * split / a.dkv_splits);
  const int n = (int)((int64_t)steps * (split + 1) / a.dkv_splits) - first;
  const int ksteps = (a.dim + 15) / 16;
  int qs = 0, gs = 0;   // the producer's: tiles of q and dO issued
  auto give_up = [&](int info) {
    *abort_flag = 1;
    if (lane == 0) report_error(&g_op_status, KFAC_ERR_TIMEOUT, -1, info);
  };
  if (warp < 4) {
  if (warp == 0) {
    if (lane == 0 && n > 0) {  // ----------------------------------------- TMA producer
      tc::mbar_expect_tx(kv_full, 2 * C::TILE);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        tc::tma_load_4d(Ks + c * kChunk, &mp.k, kv_full, 64 * c, k0, hk * mp.xk.head, b * mp.xk.batch);
        tc::tma_load_4d(Vs + c * kChunk, &mp.v, kv_full, 64 * c, k0, hk * mp.xv.head, b * mp.xv.batch);
      }
      for (int i = 0; i < n; ++i) {
        const int h = hk * a.group + (first + i) / qtiles, row = (first + i) % qtiles * BT;
        const int sq = i % 3, sg = i % 2;
        if (!tc::mbar_wait(&q_empty[sq], ((uint32_t)(i / 3) & 1u) ^ 1u, abort_flag)) break;
        load_chunks<NC>(Qs + sq * C::TILE, &mp.q, &q_full[sq], row, h * mp.xq.head, b * mp.xq.batch);
        ++qs;
        if (!tc::mbar_wait(&g_empty[sg], ((uint32_t)(i / 2) & 1u) ^ 1u, abort_flag)) break;
        load_chunks<NC>(Gs + sg * C::TILE, &mp.g, &g_full[sg], row, h * mp.xg.head, b * mp.xg.batch);
        ++gs;
      }
      if (gs < n) give_up(111);
    }
  } else if (warp == 1) {
    if (n > 0) {  // ------------------------------------------------------- MMA issuer
      const uint32_t leader = tc::elect_leader();
      const uint32_t idesc = tc::make_idesc(1, 128, ksteps * 16) | tc::kIdescMnB;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = __all_sync(kFull, tc::mbar_wait(bar, parity, abort_flag));
        if (!ok) give_up(112);
        return ok;
      };
      bool ok = wait(kv_ready, 0) && wait(&q_full[0], 0);
      if (ok) {
        mma_scores(leader, s_at(0), Ks, Qs, ksteps);
        tc::umma_commit_by(leader, s_full(0));
      }
      for (int i = 0; i < n && ok; ++i) {
        const int sq = i % 3, sg = i % 2, s1 = (i + 1) % 3;
        const uint32_t ph = (uint32_t)i & 1u;
        if (!(ok = wait(&g_full[sg], (uint32_t)(i / 2) & 1u))) break;
        mma_scores(leader, tmem + 128, Vs, Gs + sg * C::TILE, ksteps);
        tc::umma_commit_by(leader, dp_full);
        auto next_scores = [&]() {
          if (i + 1 == n) return true;
          if (!wait(&q_full[s1], (uint32_t)((i + 1) / 3) & 1u)) return false;
          mma_scores(leader, s_at(i + 1), Ks, Qs + s1 * C::TILE, ksteps);
          tc::umma_commit_by(leader, s_full(i + 1));
          return true;
        };
        if (NC == 1 && !(ok = next_scores())) break;
        if (!(ok = wait(p_ready, ph))) break;
        tc::tc_fence_after();
        for (int u = 0; u < 2; ++u)
          mma_values(leader, tmem + 256, s_at(i) + 64 * u, Gs + sg * C::TILE + u * kHalf, idesc, i > 0 || u > 0);
        tc::umma_commit_by(leader, &g_empty[sg]);
        if (NC == 2 && !(ok = next_scores())) break;
        if (!(ok = wait(ds_ready, ph))) break;
        tc::tc_fence_after();
        for (int u = 0; u < 2; ++u)
          mma_values(leader, tmem + 256 + 64 * NC, tmem + 128 + 64 * u, Qs + sq * C::TILE + u * kHalf, idesc, i > 0 || u > 0);
        tc::umma_commit_by(leader, &q_empty[sq]);
      }
      if (ok) tc::umma_commit_by(leader, done);
    }
  } else if (warp == 2) {  // ------------------------- keys not permitted, row statistics
    // Their rows of K and V become zero, so that whatever stands there cannot make an
    // exception of its lane; the lane's own results are dropped at the end.
    if (n > 0) {
      uint32_t w[4];
      MaskWalk mask;
      mask.fetch(a, b, len, k0);
      mask.words(a, len, k0, w);
      if (__all_sync(kFull, tc::mbar_wait(kv_full, 0, abort_flag))) {
        if (!all_ok(w)) {
          zero_rows<NC>(Ks, w);
          zero_rows<NC>(Vs, w);
        }
        if (lane == 0) tc::mbar_arrive(kv_ready);
      } else {
        give_up(113);
      }
    }
    for (int i = 0; i < n; ++i) {
      const int h = hk * a.group + (first + i) / qtiles, row = (first + i) % qtiles * BT, s = i % 2;
      if (!__all_sync(kFull, tc::mbar_wait(&st_empty[s], ((uint32_t)(i / 2) & 1u) ^ 1u, abort_flag))) {
        give_up(113);
        break;
      }
      const int64_t at = ((int64_t)b * a.heads + h) * a.len_q + row;
      float* dst = stats + s * 2 * BT;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int r = 32 * c + lane;
        const bool in = row + r < a.len_q;
        // negated; past the queries, or a query without keys: P = exp(S - inf) = 0
        const float z = in ? -__ldg(a.lse_in + at + r) * kLog2e : -INFINITY;
        dst[r] = z == INFINITY ? -INFINITY : z;
        dst[BT + r] = in ? -a.delta[at + r] : 0.f;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&st_full[s]);
    }
  }
  } else {  // ----------------------------------------------- P^T and dS^T
    const int half = (warp - 4) / 4;   // columns [64 half, 64 half + 64)
    const uint32_t lanes = (uint32_t)(warp % 4) * 32 << 16;
    const uint32_t td = tmem + lanes + 128 + 64 * half;
    const int key = k0 + 32 * (warp % 4) + lane;
    const bool mine = key_ok(a, b, len, key);
    const bool one = one_key(a, b, len);   // while the first tiles are on their way
    const float c2 = a.scale * kLog2e;
    const F2 cc2 = f2(c2, c2);
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const uint32_t ph = (uint32_t)i & 1u;
      const int s = i % 2;
      const float4* lse = reinterpret_cast<const float4*>(stats + s * 2 * BT + 64 * half);
      const float4* delta = lse + BT / 4;
      ok = __all_sync(kFull, tc::mbar_wait(&st_full[s], (uint32_t)(i / 2) & 1u, abort_flag) &&
                                 tc::mbar_wait(s_full(i), s_phase(i), abort_flag));
      if (!ok) break;
      tc::tc_fence_after();
      const uint32_t ts = s_at(i) + lanes + 64 * half;
      uint32_t r[2][32];
      tc::tmem_ld32_issue(ts, r[0]);
      tc::tmem_ld32_issue(ts + 32, r[1]);
      tc::tmem_ld_wait();
      tc::tmem_ld_use(r[0]);
      tc::tmem_ld_use(r[1]);
      F2 p[32];
      uint32_t u[32];
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        const float4 z = lse[c / 2];   // negated
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i2 = 2 * (c + e);
          float x, y;
          unpack(fma2(f2(r[i2 / 32][i2 % 32], r[i2 / 32][i2 % 32 + 1]), cc2, e ? f2(z.z, z.w) : f2(z.x, z.y)),
                 &x, &y);
          x = ex2(x);
          y = ex2(y);
          p[c + e] = f2(x, y);
          u[c + e] = pack_bf16(x, y);
        }
      }
      tc::tmem_st32(ts, u);
      tc::tmem_st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(p_ready);
      ok = __all_sync(kFull, tc::mbar_wait(dp_full, ph, abort_flag));
      if (!ok) break;
      tc::tc_fence_after();
      tc::tmem_ld32_issue(td, r[0]);
      tc::tmem_ld32_issue(td + 32, r[1]);
      tc::tmem_ld_wait();
      tc::tmem_ld_use(r[0]);
      tc::tmem_ld_use(r[1]);
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        const float4 z = delta[c / 2];   // negated
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i2 = 2 * (c + e);
          float x, y;
          unpack(mul2(p[c + e], add2(f2(r[i2 / 32][i2 % 32], r[i2 / 32][i2 % 32 + 1]),
                                     e ? f2(z.z, z.w) : f2(z.x, z.y))), &x, &y);
          u[c + e] = pack_bf16(x, y);
        }
      }
      tc::tmem_st32(td, u);
      tc::tmem_st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&st_empty[s]);
        tc::mbar_arrive(ds_ready);
      }
    }
    if (n > 0 && ok) ok = __all_sync(kFull, tc::mbar_wait(done, 0, abort_flag));
    if (!ok) give_up(114);
    tc::tc_fence_after();
    // dV by the first group, dK by the second
    const int64_t* st = half ? a.dks : a.dvs;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(half ? a.dk : a.dv) + b * st[0] + key * st[1] + hk * st[2];
    const float f = !ok ? kNaN : half ? a.scale : 1.f;
    const bool zero = n == 0 || !mine || (half && one);
    float* part = (half ? a.part_dk : a.part_dv) +
                  ((((int64_t)split * a.batch + b) * a.kv_heads + hk) * a.len_kv + key) * a.dim;
    for (int c = 0; c < a.dim; c += 32) {
      uint32_t o[32];
      if (n > 0) {
        tc::tmem_ld32_issue(tmem + lanes + 256 + 64 * NC * half + c, o);
        tc::tmem_ld_wait();
        tc::tmem_ld_use(o);
      }
      if (key >= a.len_kv) continue;
      if (a.dkv_splits == 1) store_row(o, dst, c, a.dim, f, zero);
      else store_part(o, part, c, a.dim, ok, zero);
    }
    tc::tc_fence_before();
  }
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) {
      land(kv_full, n > 0);
      land_ring<3>(q_full, qs);
      land_ring<2>(g_full, gs);
    }
    if (warp == 1) end_mmas(ended);
    __syncthreads();
  }
}

template <int NC>
__device__ __forceinline__ void dq_block(const Args& a, const BwdMaps& mp, int tile, int split, int hk, int b, uint8_t* smem,
                                         uint64_t* bars, volatile int* abort_flag, uint32_t tmem) {
  using C = BwdCfg<NC>;
  uint8_t *Qs = smem, *Gs = Qs + C::TILE, *Ks = Gs + C::TILE, *Vs = Ks + 3 * C::TILE;
  uint64_t *qg_full = bars, *k_full = bars + 1, *k_empty = bars + 4, *v_full = bars + 7,
           *v_empty = bars + 9, *dp_full = bars + 11, *s_read = bars + 13, *ds_ready = bars + 14,
           *s_full = bars + 15, *ended = bars + 16, *done = bars + 19, *k_ready = bars + 20,
           *w_full = bars + 23;
  uint4* words = reinterpret_cast<uint4*>(bars + 28);   // [3] permitted keys of a tile
  const int warp = __shfl_sync(kFull, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int qtiles = (a.len_q + BT - 1) / BT;
  const int h = hk * a.group + tile / qtiles, q0 = tile % qtiles * BT;
  const int len = __shfl_sync(kFull, walk_end(a, b), 0);   // known to be warp-uniform
  // this part of the key tiles
  const int tiles = (len + BT - 1) / BT;
  const int first = (int)((int64_t)tiles * split / a.dq_splits);
  const int n = (int)((int64_t)tiles * (split + 1) / a.dq_splits) - first;
  const int ksteps = (a.dim + 15) / 16;
  int ks = 0, vs = 0;   // the producer's: tiles of k and v issued
  auto give_up = [&](int info) {
    *abort_flag = 1;
    if (lane == 0) report_error(&g_op_status, KFAC_ERR_TIMEOUT, -1, info);
  };
  if (warp < 4) {
  if (warp == 0) {
    if (lane == 0 && n > 0) {  // ----------------------------------------- TMA producer
      tc::mbar_expect_tx(qg_full, 2 * C::TILE);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        tc::tma_load_4d(Qs + c * kChunk, &mp.q, qg_full, 64 * c, q0, h * mp.xq.head, b * mp.xq.batch);
        tc::tma_load_4d(Gs + c * kChunk, &mp.g, qg_full, 64 * c, q0, h * mp.xg.head, b * mp.xg.batch);
      }
      for (int j = 0; j < n; ++j) {
        const int sk = j % 3, sv = j % 2;
        if (!tc::mbar_wait(&k_empty[sk], ((uint32_t)(j / 3) & 1u) ^ 1u, abort_flag)) break;
        load_chunks<NC>(Ks + sk * C::TILE, &mp.k, &k_full[sk], (first + j) * BT, hk * mp.xk.head, b * mp.xk.batch);
        ++ks;
        if (!tc::mbar_wait(&v_empty[sv], ((uint32_t)(j / 2) & 1u) ^ 1u, abort_flag)) break;
        load_chunks<NC>(Vs + sv * C::TILE, &mp.v, &v_full[sv], (first + j) * BT, hk * mp.xv.head, b * mp.xv.batch);
        ++vs;
      }
      if (vs < n) give_up(121);
    }
  } else if (warp == 1) {
    if (n > 0) {  // ------------------------------------------------------- MMA issuer
      const uint32_t leader = tc::elect_leader();
      const uint32_t idesc = tc::make_idesc(1, 128, ksteps * 16) | tc::kIdescMnB;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = __all_sync(kFull, tc::mbar_wait(bar, parity, abort_flag));
        if (!ok) give_up(122);
        return ok;
      };
      auto scores = [&](int j) {
        const int s = j % 3;
        if (!wait(&k_ready[s], (uint32_t)(j / 3) & 1u)) return false;
        mma_scores(leader, tmem, Qs, Ks + s * C::TILE, ksteps);
        tc::umma_commit_by(leader, s_full);
        return true;
      };
      auto grads = [&](int j) {
        const int s = j % 2;
        if (!wait(&v_full[s], (uint32_t)(j / 2) & 1u)) return false;
        mma_scores(leader, tmem + 128 + 128 * (j % 2), Gs, Vs + s * C::TILE, ksteps);
        tc::umma_commit_by(leader, &dp_full[j % 2]);
        tc::umma_commit_by(leader, &v_empty[s]);
        return true;
      };
      bool ok = wait(qg_full, 0) && scores(0) && grads(0);
      for (int j = 0; j < n && ok; ++j) {
        if (j + 1 < n) {   // S has been read; dS(j - 1), in dP's other buffer, multiplied
          if (!(ok = wait(s_read, (uint32_t)j & 1u))) break;
          tc::tc_fence_after();
          if (!(ok = scores(j + 1) && grads(j + 1))) break;
        }
        if (!(ok = wait(ds_ready, (uint32_t)j & 1u))) break;
        tc::tc_fence_after();
        for (int u = 0; u < 2; ++u)
          mma_values(leader, tmem + 384, tmem + 128 + 128 * (j % 2) + 64 * u, Ks + j % 3 * C::TILE + u * kHalf,
                     idesc, j > 0 || u > 0);
        tc::umma_commit_by(leader, &k_empty[j % 3]);
        if (j + 1 == n) tc::umma_commit_by(leader, done);
      }
    }
  } else if (warp == 2) {  // ----------------------------------------------- key mask
    // K's rows of keys that are not permitted become zero: dS is 0 there, and 0 x NaN
    // would reach dQ
    MaskWalk mask;
    mask.fetch(a, b, len, first * BT);
    for (int j = 0; j < n; ++j) {
      const int s = j % 3;
      uint32_t w[4];
      mask.words(a, len, (first + j) * BT, w);
      mask.fetch(a, b, len, (first + j + 1) * BT);
      // the slot's last tile has been multiplied, so its words have been read
      bool ok = tc::mbar_wait(&k_empty[s], ((uint32_t)(j / 3) & 1u) ^ 1u, abort_flag);
      if (ok && lane == 0) {
        words[s] = make_uint4(w[0], w[1], w[2], w[3]);
        tc::mbar_arrive(&w_full[s]);
      }
      ok = __all_sync(kFull, ok && tc::mbar_wait(&k_full[s], (uint32_t)(j / 3) & 1u, abort_flag));
      if (!ok) {
        give_up(123);
        break;
      }
      if (!all_ok(w)) zero_rows<NC>(Ks + s * C::TILE, w);
      if (lane == 0) tc::mbar_arrive(&k_ready[s]);
    }
  }
  } else {  // -------------------------------------------------------- dS
    const int half = (warp - 4) / 4;   // columns [64 half, 64 half + 64)
    const uint32_t lanes = (uint32_t)(warp % 4) * 32 << 16;
    const uint32_t ts = tmem + lanes + 64 * half;
    const int q = q0 + 32 * (warp % 4) + lane;
    const int64_t row = ((int64_t)b * a.heads + h) * a.len_q + q;
    const bool in = q < a.len_q;
    float lse = in ? __ldg(a.lse_in + row) * kLog2e : INFINITY;
    if (lse == -INFINITY) lse = INFINITY;   // no permitted key: P = 0
    const float delta = in ? a.delta[row] : 0.f;
    const bool one = one_key(a, b, len);   // while the first tiles are on their way
    const float c2 = a.scale * kLog2e;
    const F2 cc2 = f2(c2, c2), nl2 = f2(-lse, -lse), nd2 = f2(-delta, -delta);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      ok = __all_sync(kFull, tc::mbar_wait(s_full, (uint32_t)j & 1u, abort_flag) &&
                                 (!a.key_mask || tc::mbar_wait(&w_full[j % 3], (uint32_t)(j / 3) & 1u,
                                                               abort_flag)));
      if (!ok) break;
      tc::tc_fence_after();
      uint32_t w[4];
      if (a.key_mask) {
        const uint4 u = words[j % 3];
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
      } else {
        len_words(len, (first + j) * BT, w);
      }
      const uint32_t td = ts + 128 + 128 * (j % 2);
      uint32_t r[2][32];
      tc::tmem_ld32_issue(ts, r[0]);
      tc::tmem_ld32_issue(ts + 32, r[1]);
      tc::tmem_ld_wait();
      tc::tmem_ld_use(r[0]);
      tc::tmem_ld_use(r[1]);
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(s_read);
      F2 p[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        float x, y;
        unpack(fma2(f2(r[c / 16][2 * c % 32], r[c / 16][2 * c % 32 + 1]), cc2, nl2), &x, &y);
        p[c] = f2(ex2(x), ex2(y));
      }
      ok = __all_sync(kFull, tc::mbar_wait(&dp_full[j % 2], (uint32_t)(j / 2) & 1u, abort_flag));
      if (!ok) break;
      tc::tc_fence_after();
      tc::tmem_ld32_issue(td, r[0]);
      tc::tmem_ld32_issue(td + 32, r[1]);
      tc::tmem_ld_wait();
      tc::tmem_ld_use(r[0]);
      tc::tmem_ld_use(r[1]);
      uint32_t u[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        float x, y;
        unpack(mul2(p[c], add2(f2(r[c / 16][2 * c % 32], r[c / 16][2 * c % 32 + 1]), nd2)), &x, &y);
        u[c] = pack_bf16(x, y);
      }
      if (!all_ok(w)) {
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const uint32_t bits = (half ? w[2 + c / 16] : w[c / 16]) >> (2 * c % 32);
          u[c] &= (bits & 1u ? 0xffffu : 0u) | (bits & 2u ? 0xffff0000u : 0u);
        }
      }
      tc::tmem_st32(td, u);
      tc::tmem_st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(ds_ready);
    }
    if (n > 0 && ok) ok = __all_sync(kFull, tc::mbar_wait(done, 0, abort_flag));
    if (!ok) give_up(124);
    tc::tc_fence_after();
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.dq) + b * a.dqs[0] + q * a.dqs[1] + h * a.dqs[2];
    const bool zero = n == 0 || one;
    float* part = a.part_dq + ((int64_t)split * a.batch * a.heads * a.len_q + row) * a.dim;
    for (int c = 32 * half; c < a.dim; c += 64) {   // the groups take 32 channels in turn
      uint32_t o[32];
      if (n > 0) {
        tc::tmem_ld32_issue(tmem + lanes + 384 + c, o);
        tc::tmem_ld_wait();
        tc::tmem_ld_use(o);
      }
      if (!in) continue;
      if (a.dq_splits == 1) store_row(o, dst, c, a.dim, ok ? a.scale : kNaN, zero);
      else store_part(o, part, c, a.dim, ok, zero);
    }
    tc::tc_fence_before();
  }
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) {
      land(qg_full, n > 0);
      land_ring<3>(k_full, ks);
      land_ring<2>(v_full, vs);
    }
    if (warp == 1) end_mmas(ended);
    __syncthreads();
  }
}

// grid: every dK/dV block, then every dQ block: the longer ones start first.
template <int NC>
__global__ void __launch_bounds__(kTcThreads, 1)
tc_backward_kernel(const __grid_constant__ Args a, const __grid_constant__ BwdMaps mp) {
  using C = BwdCfg<NC>;
  extern __shared__ __align__(1024) uint8_t smem[];   // the 128-byte swizzle's period
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + 7 * C::TILE + C::STATS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBwdBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = __shfl_sync(kFull, (int)threadIdx.x / 32, 0);
  const int key_tiles = (a.len_kv + BT - 1) / BT, q_tiles = a.group * ((a.len_q + BT - 1) / BT);
  const int dkv_blocks = key_tiles * a.dkv_splits * a.kv_heads * a.batch;
  const bool dkv = (int)blockIdx.x < dkv_blocks;
  const int id = dkv ? (int)blockIdx.x : (int)blockIdx.x - dkv_blocks;
  const int tiles = dkv ? key_tiles : q_tiles, splits = dkv ? a.dkv_splits : a.dq_splits;
  const int tile = id % tiles, split = id / tiles % splits, pair = id / tiles / splits;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBwdBars; ++i) {
      // 13: p_ready or s_read, 14: ds_ready (one arrival per warp of the two groups);
      // 17, 18: the dK/dV role's st_empty (the same)
      const bool warps = i == 13 || i == 14 || i == 17 || i == 18;
      tc::mbar_init(&bars[i], warps ? 8 : 1);
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
  const uint32_t tmem = __shfl_sync(kFull, *tmem_slot, 0);
  pdl_wait();
  pdl_trigger();
  if (dkv) dkv_block<NC>(a, mp, tile, split, pair % a.kv_heads, pair / a.kv_heads, smem, bars, abort_flag, tmem);
  else dq_block<NC>(a, mp, tile, split, pair % a.kv_heads, pair / a.kv_heads, smem, bars, abort_flag, tmem);
  if (warp == 1) tc::tmem_dealloc(tmem, 512);   // (both end behind a barrier)
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

template <int NC, int NT>
kfac_status launch_tc_forward(const Args& a, cudaStream_t st) {
  using C = FwdCfg<NC, NT>;
  static OncePerDevice once;
  const kfac_status e = allow_smem(once, tc_forward_kernel<NC, NT>, C::SMEM);
  if (e != KFAC_OK) return e;
  CUtensorMap mq, mk, mv;
  MapMul xq, xk, xv;
  if (!make_map(&mq, &xq, a.q, a.qs, a.dim, a.len_q, a.heads, a.batch) ||
      !make_map(&mk, &xk, a.k, a.ks, a.dim, a.len_kv, a.kv_heads, a.batch) ||
      !make_map(&mv, &xv, a.v, a.vs, a.dim, a.len_kv, a.kv_heads, a.batch))
    return KFAC_ERR_CUDA;
  const dim3 grid((unsigned)(cdiv(a.len_q, NT * BT) * a.splits), a.heads, a.batch);
  launch_pdl(tc_forward_kernel<NC, NT>, grid, dim3(C::THREADS), C::SMEM, st, a, mq, mk, mv, xq, xk, xv);
  count_launch();
  return check_launch();
}

template <int NC>
kfac_status launch_tc_backward(const Args& a, cudaStream_t st) {
  using C = BwdCfg<NC>;
  static OncePerDevice once;
  const kfac_status e = allow_smem(once, tc_backward_kernel<NC>, C::SMEM);
  if (e != KFAC_OK) return e;
  BwdMaps m;
  if (!make_map(&m.q, &m.xq, a.q, a.qs, a.dim, a.len_q, a.heads, a.batch) ||
      !make_map(&m.k, &m.xk, a.k, a.ks, a.dim, a.len_kv, a.kv_heads, a.batch) ||
      !make_map(&m.v, &m.xv, a.v, a.vs, a.dim, a.len_kv, a.kv_heads, a.batch) ||
      !make_map(&m.g, &m.xg, a.dout, a.dos, a.dim, a.len_q, a.heads, a.batch))
    return KFAC_ERR_CUDA;
  const int64_t blocks = (cdiv(a.len_kv, BT) * a.dkv_splits + a.group * cdiv(a.len_q, BT) * a.dq_splits) *
                         a.kv_heads * a.batch;
  if (blocks > INT32_MAX) return KFAC_ERR_INVALID_ARG;
  const dim3 grid((unsigned)blocks);
  launch_pdl(tc_backward_kernel<NC>, grid, dim3(kTcThreads), C::SMEM, st, a, m);
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

// Query tiles per block.  One (two blocks per SM) up to 64 channels, where the
// exponentials bound the kernel and two independent blocks hide each other's chains (2 x
// 2432 queries, 4096 ragged keys, 16 heads x 64: 73 us, with two tiles 105 us), and where a
// block's walk is short and its set-up and end weigh (14 x 316 queries, 35 keys, 32 heads x 128:
// 42 us against 50 us).  Two where the products bound it and share each tile of keys (8 x 2048
// queries, 4096 ragged keys, 16 heads x 128: 222 us against 242 us; 4 x 1000 queries, 8192 keys:
// 141 us against 156 us).  (Times with a flushed L2.)
int tc_forward_tiles(int dim, int len_q, int len_kv) {
  return dim <= 64 || len_q <= BT || len_kv <= 2 * BT ? 1 : 2;
}

kfac_status tc_forward(const Args& a, cudaStream_t st) {
  if (a.dim <= 64) return launch_tc_forward<1, 1>(a, st);
  return tc_forward_tiles(a.dim, a.len_q, a.len_kv) == 1 ? launch_tc_forward<2, 1>(a, st)
                                                         : launch_tc_forward<2, 2>(a, st);
}

bool tc_backward_ok(const Args& a) {
  return a.dim % 8 == 0 && a.len_q > 0 && a.len_kv > 0 &&
         rows_ok(a.q, a.qs, a.len_q, a.heads, a.batch) &&
         rows_ok(a.k, a.ks, a.len_kv, a.kv_heads, a.batch) &&
         rows_ok(a.v, a.vs, a.len_kv, a.kv_heads, a.batch) &&
         rows_ok(a.dout, a.dos, a.len_q, a.heads, a.batch) &&
         rows_ok(a.dq, a.dqs, a.len_q, a.heads, a.batch) &&
         rows_ok(a.dk, a.dks, a.len_kv, a.kv_heads, a.batch) &&
         rows_ok(a.dv, a.dvs, a.len_kv, a.kv_heads, a.batch);
}

kfac_status tc_backward(const Args& a, cudaStream_t st) {
  return a.dim <= 64 ? launch_tc_backward<1>(a, st) : launch_tc_backward<2>(a, st);
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
