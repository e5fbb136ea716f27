// Matrices whose smaller side is at most 128: all steps of one in one launch, X in shared memory.
// Included by k_ortho.cu, inside its namespace.
//
// A matrix takes a cluster of 1, 2, 4 or 8 blocks; block b holds its columns (rows of a tall
// matrix: X is G^T then) [b w, (b + 1) w) as an fp16 tile of 128 rows, padded with zeros.  Per step:
//   L = X X^T      one 128 x 128 tcgen05 product per block; the blocks' parts are added in fp32 through
//                  distributed shared memory, each block a share of the columns, in the blocks' order
//   M = a I + b L + c L^2   by every block
//   X <- M X       by every block, its columns (X is the K-major operand above and, as it lies, the
//                  MN-major one here)
// What bounds it is the chain: three products, three passes through TMEM and registers and, with
// several blocks, two cluster barriers per step.  A product launch per step and product (the
// large matrices' form) pays 6 to 8 us for each.

constexpr int kSide = 128;
constexpr int kSmallThreads = 512;                // 16 warps: four for each quarter of TMEM's lanes
constexpr int kSmallTasks = 64;                  // matrices per launch
constexpr int kTileBytes = kSide * 64 * 2;       // 128 rows x 64 columns

struct SmallTask {
  PrepTask in;                                   // (x, m and their layout alone)
  void* out;                                     // the direction or the weights
  int64_t ldo;
  float rate;
};
struct SmallStep {
  float gram, poly, beta, diag, apply;
  int shift_in, shift_out;                       // of X before and after the step, see Plan
};
struct SmallLaunch {
  SmallTask task[kSmallTasks];
  SmallStep step[kMaxSteps];
  int steps, cluster, tiles;                     // tiles: of 64 columns per block
  int nesterov;
  int give_up;                                   // self-test: a step whose first wait counts as one that ran out
  float mu, keep;
  double eps;
};

template <bool kFull> struct SmallCfg {
  static constexpr int HALVES = kFull ? 2 : 1;
  // columns per block: what shared memory holds beside L (or M) and, in a cluster, the parts of L
  // (full arithmetic: and TMEM, 128 columns for each tile's part of L)
  static constexpr int most_tiles(int cluster) { return kFull ? (cluster > 1 ? 3 : 4) : 8; }
  static constexpr size_t smem(int tiles, int cluster) {
    const size_t bytes = (size_t)HALVES * (tiles + 2) * kTileBytes + (cluster > 1 ? kSide * kSide * 4 : 0);
    return 1024 + (bytes < kSmallThreads * 128 ? kSmallThreads * 128 : bytes);   // (4 KB a warp at the end)
  }
  static_assert(smem(most_tiles(1), 1) <= 231424 && smem(most_tiles(8), 8) <= 231424, "shared memory");
};

__device__ __forceinline__ void st_cluster_f4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d)
               : "memory");
}
__device__ __forceinline__ void st_cluster_u2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
// Offset of (row, column) in tiles of 128 rows x 64 columns, 128-byte swizzle.
__device__ __forceinline__ int tile_offset(int row, int col) {
  return (col >> 6) * kTileBytes + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4) + (col & 7) * 2;
}

template <int TO, typename TI, typename T, bool kFull>
__global__ void __launch_bounds__(kSmallThreads, 1) ortho_small_kernel(const __grid_constant__ SmallLaunch g) {
  constexpr bool kStep = TO == TO_WEIGHTS;
  constexpr int HALVES = kFull ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t done;
  __shared__ uint32_t tmem_slot, lost;   // lost: a block of the cluster gave up
  __shared__ float red[3][kSmallThreads / 32];
  __shared__ float parts[8][3], factors[4];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* const xs = smem;                                            // [halves][tiles]
  uint8_t* const ls = xs + (size_t)HALVES * g.tiles * kTileBytes;      // [halves][2]: L, then M
  float* const recv = reinterpret_cast<float*>(ls + HALVES * 2 * kTileBytes);   // [src][column / 4][row][4]
  const int x_lo = g.tiles * kTileBytes, l_lo = 2 * kTileBytes;        // from a hi tile to its lo tile
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cs = g.cluster, rank = (int)(blockIdx.x % cs);
  const SmallTask& task = g.task[blockIdx.x / cs];
  const PrepTask& t = task.in;
  const bool tall = t.rows > t.cols;
  const int s = tall ? t.cols : t.rows, l = tall ? t.rows : t.cols;
  const int l0 = rank * g.tiles * 64, width = max(0, min(l - l0, g.tiles * 64));
  const int used = (width + 63) / 64;                                  // tiles with columns
  auto cluster_sync = [&]() {
    if (cs > 1) tc::cluster_sync();
    else __syncthreads();
  };

  if (threadIdx.x == 0) {
    tc::mbar_init(&done, 1);
    lost = 0;
    tc::fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc(&tmem_slot, 512);
    tc::tmem_relinquish();
  }
  for (int i = threadIdx.x; i < HALVES * g.tiles * kTileBytes / 16; i += kSmallThreads)
    reinterpret_cast<uint4*>(xs)[i] = make_uint4(0u, 0u, 0u, 0u);
  tc::tc_fence_before();
  cluster_sync();   // (a block's shared memory is written to by the others only once it has started)
  tc::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();
  pdl_trigger();
  bool ok = true;
  uint32_t phase = 0;

  // ------------------------------------------------------------------ norm, X_0
  // f(row of X, column of X in this block, values) for this block's part of the matrix; values run
  // along the columns of X, or (tall) along its rows
  auto visit = [&](auto n_, auto fresh, auto f) {
    constexpr int N = decltype(n_)::value;
    const int per = ((tall ? s : width) + N - 1) / N;
    const int total = per * (tall ? width : s);
    constexpr int AHEAD = N == 1 ? 16 : 4;   // loads in flight
    for (int i = threadIdx.x; i < total; i += AHEAD * kSmallThreads) {
      Piece<TI, N, kStep> p[AHEAD];
      int row[AHEAD], c[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int at = i + k * kSmallThreads;
        if (at >= total) continue;
        row[k] = at / per;
        c[k] = (at - row[k] * per) * N;
        p[k].load(t, row[k] + (tall ? l0 : 0), c[k] + (tall ? 0 : l0));
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        if (i + k * kSmallThreads >= total) continue;
        float u[N];
        p[k].template use<decltype(fresh)::value>(g.mu, g.nesterov, t, row[k] + (tall ? l0 : 0),
                                                  c[k] + (tall ? 0 : l0), u);
        f(row[k], c[k], u);
      }
    }
  };
  auto visit_by = [&](auto fresh, auto f) {
    if (t.vec) visit(std::integral_constant<int, 16 / (int)sizeof(TI)>(), fresh, f);
    else visit(std::integral_constant<int, 1>(), fresh, f);
  };
  // The values are kept as they were read where a tile has the bits for them (bf16 in one half, fp32
  // in two), and converted in place once the norm is known; fp32 in half arithmetic is read again.
  constexpr bool kKeep = !kStep && (sizeof(TI) == 2 || kFull);
  auto put = [&](int row, int c, auto& hi, auto& lo) {   // one or more 16-bit values from (row, c) on
    constexpr int n = sizeof(hi) / 2;
    if (!tall) {
      *reinterpret_cast<Vec<uint16_t, n>*>(xs + tile_offset(row, c)) = hi;
      if (kFull) *reinterpret_cast<Vec<uint16_t, n>*>(xs + x_lo + tile_offset(row, c)) = lo;
    } else {
#pragma unroll
      for (int i = 0; i < n; ++i) {
        *reinterpret_cast<uint16_t*>(xs + tile_offset(c + i, row)) = hi.v[i];
        if (kFull) *reinterpret_cast<uint16_t*>(xs + x_lo + tile_offset(c + i, row)) = lo.v[i];
      }
    }
  };
  float up0, up1;
  bool far;             // below eps: j > 0
  {
    Squares sq;
    visit_by(std::true_type(), [&](int row, int c, auto& u) {
      sq.add(u);
      if constexpr (kKeep) {
        constexpr int n = sizeof(u) / sizeof(float);
        Vec<uint16_t, n> hi, lo;
#pragma unroll
        for (int i = 0; i < n; ++i) {
          hi.v[i] = (uint16_t)(__float_as_uint(u[i]) >> 16);
          lo.v[i] = (uint16_t)__float_as_uint(u[i]);
        }
        put(row, c, hi, lo);
      }
    });
    if (sq.unsafe()) visit_by(std::false_type(), [&](int, int, auto& u) { sq.add_scaled(u); });
    float v[3];
    sq.finish(v);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
      if (lane == 0) red[k][warp] = v[k];
    }
    __syncthreads();
    if (threadIdx.x < 3) {
      float sum = 0.f;
      for (int w = 0; w < kSmallThreads / 32; ++w) sum += red[threadIdx.x][w];
      for (int c = 0; c < cs; ++c)   // to every block of the cluster
        tc::st_cluster_u32(tc::mapa(&parts[rank][threadIdx.x], (uint32_t)c), __float_as_uint(sum));
    }
    cluster_sync();
    if (threadIdx.x == 0) {   // (64-bit arithmetic is slow: 512 threads took 7 us over it)
      double sums[3] = {0.0, 0.0, 0.0};
      for (int c = 0; c < cs; ++c)
        for (int k = 0; k < 3; ++k) sums[k] += (double)parts[c][k];
      float up[2];
      scale_factors(sums, g.eps, up, &factors[2], &factors[3]);
      factors[0] = up[0];
      factors[1] = up[1];
    }
    __syncthreads();
    up0 = factors[0];
    up1 = factors[1];
    far = factors[3] > 0.f;
  }
  auto halves_of = [&](float x, uint16_t& hi, uint16_t& lo) {
    const float v = x * up0 * up1;
    const __half h = __float2half_rn(v);
    hi = __half_as_ushort(h);
    if (kFull) lo = __half_as_ushort(__float2half_rn(v - __half2float(h)));
  };
  if constexpr (kKeep) {
    for (int i = threadIdx.x; i < used * kTileBytes / 16; i += kSmallThreads) {
      Vec<uint16_t, 8>* at = reinterpret_cast<Vec<uint16_t, 8>*>(xs) + i;
      Vec<uint16_t, 8>* at_lo = reinterpret_cast<Vec<uint16_t, 8>*>(xs + x_lo) + i;
      Vec<uint16_t, 8> hi = *at, lo;
      if (kFull) lo = *at_lo;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        halves_of(__uint_as_float((uint32_t)hi.v[j] << 16 | (kFull ? lo.v[j] : 0u)), hi.v[j], lo.v[j]);
      *at = hi;
      if (kFull) *at_lo = lo;
    }
  } else {
    visit_by(std::false_type(), [&](int row, int c, auto& u) {
      constexpr int n = sizeof(u) / sizeof(float);
      Vec<uint16_t, n> hi, lo;
#pragma unroll
      for (int i = 0; i < n; ++i) halves_of(u[i], hi.v[i], lo.v[i]);
      put(row, c, hi, lo);
    });
  }

  // --------------------------------------------------------------------- steps
  const uint32_t xa = tc::smem_u32(xs), la = tc::smem_u32(ls);
  // what the threads wrote is visible to the tensor core, and what they read of TMEM may go; then
  // warp 0 issues (one lane) and waits for the products, the others at the block's barrier
  auto products = [&](auto issue, bool quit = false) {
    tc::fence_proxy_async();
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 0 && ok) {
      tc::tc_fence_after();
      const uint32_t leader = tc::elect_leader();
      issue(leader);
      tc::umma_commit_by(leader, &done);
      __syncwarp();
      volatile int never = 0;
      if (quit || !tc::mbar_wait(&done, phase, &never)) {
        if (leader) report_error(&g_status, KFAC_ERR_TIMEOUT, -1, 46);
        ok = tc::mbar_wait(&done, phase, &never) && false;   // (TMEM goes after the products, if they end)
      }
      ok = __all_sync(0xffffffffu, ok);
      phase ^= 1;
    }
    ok = __syncthreads_and(ok);   // all give up together, and go on to the barriers without products
    tc::tc_fence_after();
  };
  constexpr uint32_t kSquare = tc::make_idesc(0, kSide, kSide);
  // hi hi, and in full arithmetic hi lo and lo hi before it
  auto mma = [&](uint32_t leader, uint32_t d, uint64_t a, uint64_t b, int a_lo, int b_lo, uint32_t idesc,
                 int pass, uint32_t acc) {
    if (!kFull || pass == 1) {
      tc::umma_f16_by(leader, d, a, b, idesc, acc);
    } else {
      tc::umma_f16_by(leader, d, a, b + (uint64_t)(b_lo >> 4), idesc, acc);
      tc::umma_f16_by(leader, d, a + (uint64_t)(a_lo >> 4), b, idesc, 1u);
    }
  };
  const int qd = warp & 3, h = warp >> 2;                  // TMEM quarter, 32 columns of L and M
  const int row = 32 * qd + lane;                          // of X, L and M
  const uint32_t lane_tmem = tmem + ((uint32_t)(32 * qd) << 16);
  // 32 values of this thread's row, columns from 32 piece on, to tiles as hi (and lo) halves
  auto store32 = [&](uint8_t* tiles, int piece, int lo, const float (&v)[32]) {
    uint8_t* at = tiles + (piece >> 1) * kTileBytes + row * 128;
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack2(v[2 * i], v[2 * i + 1]);
#pragma unroll
    for (int half = 0; half < HALVES; ++half) {
      if (half) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 hi = unpack2(w[i]);
          w[i] = pack2(v[2 * i] - hi.x, v[2 * i + 1] - hi.y);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(at + half * lo + ((((piece & 1) * 4 + j) ^ (row & 7)) << 4)) =
            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    }
  };
  // 32 columns of this thread's row of an accumulator.  Full arithmetic has one for every 64 k
  // (`parts` of them, `apart` columns), added here: in one for all of L's k it was 3.9e-6 off.
  auto load32 = [&](int col, int apart, int parts, float (&v)[32]) {
    if (parts == 0) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.f;
      return;
    }
    tc::tmem_ld32(lane_tmem + (uint32_t)col, v);
    if constexpr (kFull) {
      for (int k = 1; k < parts; ++k) {
        float w[32];
        tc::tmem_ld32(lane_tmem + (uint32_t)(col + k * apart), w);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] += w[i];
      }
    }
  };
  const int k16 = (s + 15) / 16;                           // of the small side
  // whether a product with M or L adds to what is in its accumulator
  auto more = [&](int k, int pass) { return (uint32_t)((kFull ? k % 4 > 0 : k > 0) || (kFull && pass == 1)); };
  for (int step = 0; step < g.steps; ++step) {
    const SmallStep p = g.step[step];
    const bool last = step + 1 == g.steps;
    // ---- L: this block's part
    products([&](uint32_t leader) {
      for (int pass = kFull ? 0 : 1; pass < 2; ++pass)
        for (int c = 0; c < used; ++c)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t a = tc::sdesc_kmajor_sw128(xa + c * kTileBytes + kk * 32);
            mma(leader, tmem + (kFull ? 128u * c : 0u), a, a, x_lo, x_lo, kSquare, pass,
                (!kFull && c > 0) || kk > 0 || (kFull && pass == 1));
          }
    }, step == g.give_up && rank == 0);
    // X is kept times 2^max(0, j + shift): see Plan (factors: r, j)
    auto scaled = [&](float by, int power, int shift_out) {
      if (step == 0) by *= power == 2 ? factors[2] * factors[2] : factors[2];
      if (!far) return by;
      const int j = (int)factors[3];
      return ldexpf(by, max(0, j + shift_out) - power * max(0, j + p.shift_in));
    };
    const float gram = scaled(p.gram, 2, kNoShift);
    float v[32];
    load32(32 * h, 128, used, v);
    if (cs == 1) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= gram;
      store32(ls, h, l_lo, v);
    } else {
      const int own = kSide / cs;                          // columns that a block adds up
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const int col = 32 * h + i, to = col / own, group = (col - to * own) / 4;
        const float* at = recv + (((rank * (own / 4) + group) * kSide) + row) * 4;
        st_cluster_f4(tc::mapa(at, (uint32_t)to), v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
      // (what a block sends after it gave up is no part of L: all give up with it)
      if (!ok && threadIdx.x < cs) tc::st_cluster_u32(tc::mapa(&lost, threadIdx.x), 1u);
      tc::cluster_sync();
      ok = ok && *static_cast<volatile uint32_t*>(&lost) == 0;
      const int mine = threadIdx.x % kSide;
      for (int group = threadIdx.x / kSide; group < own / 4; group += kSmallThreads / kSide) {
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < cs; ++c) {
          const float4 q = *reinterpret_cast<const float4*>(
              recv + (((c * (own / 4) + group) * kSide) + mine) * 4);
          sum.x += q.x;
          sum.y += q.y;
          sum.z += q.z;
          sum.w += q.w;
        }
        const float q[4] = {sum.x * gram, sum.y * gram, sum.z * gram, sum.w * gram};
        const uint32_t a = pack2(q[0], q[1]), b = pack2(q[2], q[3]);
        uint8_t* at = ls + tile_offset(mine, rank * own + group * 4);
        for (int c = 0; c < cs; ++c) st_cluster_u2(tc::mapa(at, (uint32_t)c), a, b);
        if constexpr (kFull) {
          const float2 ha = unpack2(a), hb = unpack2(b);
          const uint32_t al = pack2(q[0] - ha.x, q[1] - ha.y), bl = pack2(q[2] - hb.x, q[3] - hb.y);
          for (int c = 0; c < cs; ++c) st_cluster_u2(tc::mapa(at + l_lo, (uint32_t)c), al, bl);
        }
      }
      // (also: every block has read its parts before the next step's arrive)
      tc::cluster_sync();
    }
    // ---- M, over L
    products([&](uint32_t leader) {
      for (int pass = kFull ? 0 : 1; pass < 2; ++pass)
        for (int k = 0; k < k16; ++k) {
          const uint64_t a = tc::sdesc_kmajor_sw128(la + (k / 4) * kTileBytes + (k % 4) * 32);
          mma(leader, tmem + (kFull ? 128u * (k / 4) : 0u), a, a, l_lo, l_lo, kSquare, pass, more(k, pass));
        }
    });
    load32(32 * h, 128, (k16 + 3) / 4, v);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= p.poly;
#pragma unroll
    for (int half = 0; half < HALVES; ++half) {
      const uint8_t* from = ls + half * l_lo + (h >> 1) * kTileBytes + row * 128;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 q = *reinterpret_cast<const uint4*>(from + ((((h & 1) * 4 + j) ^ (row & 7)) << 4));
        const uint32_t e[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack2(e[i]);
          v[8 * j + 2 * i] = fmaf(p.beta, f.x, v[8 * j + 2 * i]);
          v[8 * j + 2 * i + 1] = fmaf(p.beta, f.y, v[8 * j + 2 * i + 1]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (32 * h + i == row) v[i] += p.diag;
    store32(ls, h, l_lo, v);
    // ---- X
    products([&](uint32_t leader) {
      for (int pass = kFull ? 0 : 1; pass < 2; ++pass)
        for (int k = 0; k < k16; ++k) {
          const uint64_t a = tc::sdesc_kmajor_sw128(la + (k / 4) * kTileBytes + (k % 4) * 32);
          for (int c = 0; c < used; c += 4) {
            const uint64_t b = tc::sdesc_mnmajor_sw128(xa + c * kTileBytes + k * 2048, kTileBytes);
            mma(leader, tmem + (uint32_t)(64 * c) + (kFull ? 256u * (k / 4) : 0u), a, b, l_lo, x_lo,
                tc::make_idesc(0, kSide, 64 * min(4, used - c)) | tc::kIdescMnB, pass, more(k, pass));
          }
        }
    });
    const float apply = scaled(p.apply, 1, p.shift_out);
    for (int piece = h; piece < 2 * used; piece += 4) {
      load32(32 * piece, 256, (k16 + 3) / 4, v);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= apply;
      if (!last) {
        store32(xs, piece, x_lo, v);
        continue;
      }
      auto emit = [&](T* at, float x) {
        if constexpr (TO == TO_WEIGHTS) {
          if (ok) *at = fmaf(-task.rate, x, g.keep * *at);
        } else {
          *at = (T)(ok ? x : __int_as_float(0x7fffffff));
        }
      };
      if (tall) {                          // lanes along the rows of out
        T* at = static_cast<T*>(task.out) + (int64_t)(l0 + 32 * piece) * task.ldo + row;
        const int n = min(32, width - 32 * piece);
        if (row < s) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i < n) emit(at + (int64_t)i * task.ldo, v[i]);
        }
      } else {   // through the space of X and M, which the products have read: rows of out in whole pieces
        float* mine = reinterpret_cast<float*>(smem) + warp * 1024;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<float4*>(mine + lane * 32 + ((j ^ (lane & 7)) << 2)) =
              make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        __syncwarp();
        const int col = 32 * piece + lane, rows = min(32, s - 32 * qd);
        T* at = static_cast<T*>(task.out) + (int64_t)(32 * qd) * task.ldo + l0 + col;
        if (col < width) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i < rows)
              emit(at + (int64_t)i * task.ldo, mine[i * 32 + (((lane >> 2) ^ (i & 7)) << 2) + (lane & 3)]);
        }
      }
    }
  }
  tc::tc_fence_before();
  cluster_sync();   // no block's shared memory goes while another may write to it
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// Blocks in a cluster for a matrix of this long side (0: too long).
template <bool kFull> int small_cluster(int l) {
  for (int cs = 1; cs <= 8; cs *= 2)
    if (l <= cs * SmallCfg<kFull>::most_tiles(cs) * 64) return cs;
  return 0;
}
