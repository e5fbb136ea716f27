// Token embedding and its gradient by sorted tokens:
//   out[t] = scale table[ids[t]];   dtable[v] = scale sum_{t: ids[t] = v} dout[t].
//
// Both are bound by memory: the forward pass reads and writes a row per token, the gradient
// reads dout once and writes the whole table (the larger part for a large vocabulary).
// The gradient needs the tokens of each row together.  They are sorted by id with a stable
// radix sort (8 bits a pass, ranks from warp ballots), so that every row is summed in the order
// of its tokens: no atomics, the same inputs give the same bits.  Up to 16384 tokens a cluster of
// eight blocks sorts through distributed shared memory while the launch's other blocks clear
// the table (one block alone took 42 us for 16384 tokens; up to 2048 one does); beyond that, histogram, scan and scatter
// launches per pass, and what is cleared are the rows without tokens, beside the joins.
// Text has hot ids (padding, articles), so the sums are divided by tokens, not by rows: a chunk of
// the sorted order per block, each run inside it to its row; a second launch joins the parts of
// runs that cross chunks, in order.
#include "kfac_internal.cuh"
#include "per_device.h"
#include "tc_prims.cuh"

#include <algorithm>
#include <cmath>

namespace kfac {
namespace {

constexpr int64_t kMaxIds = (int64_t(1) << 31) - 2;
constexpr int kSmallTokens = 16384;    // sorted by one cluster
constexpr int kCluster = 8, kSortThreads = 512;
constexpr int kTileThreads = 256, kTileItems = 4096;   // of the launches per pass beyond that
constexpr int kBits = 8, kDigits = 1 << kBits;

struct EmbedArgs {
  const void* ids;
  const void* src;         // table (forward) or dout (backward)
  void* out;               // out (forward)
  float* dtable;
  float* frequency;
  int64_t tokens, rows, width, ld_src, ld_out;   // ld_out: of out or of dtable
  int64_t padding_id;
  float scale, inv_tokens;
  int id64, accumulate, passes;
  // sorted order: keys and tokens; where each row's run starts and ends
  uint32_t *keys, *vals, *keys2, *vals2;
  uint32_t *start, *end;
  uint32_t *hist, *total;  // [kDigits][tiles], [kDigits]
  int tiles;
  float* part;             // [chunks][2][width]
  int chunk;
  int late;                // rows without tokens are cleared after the sums, not all rows before them
};

template <typename T, int N> struct alignas(N * sizeof(T)) Vec { T v[N]; };

__device__ __forceinline__ int64_t id_at(const EmbedArgs& a, int64_t t) {
  return a.id64 ? __ldg(static_cast<const long long*>(a.ids) + t)
                : (int64_t)__ldg(static_cast<const int*>(a.ids) + t);
}
// The sort's key: a row, or `rows` for tokens that no row sums.
__device__ __forceinline__ uint32_t key_at(const EmbedArgs& a, int64_t t) {
  const int64_t id = id_at(a, t);
  return id >= 0 && id < a.rows && id != a.padding_id ? (uint32_t)id : (uint32_t)a.rows;
}

// ------------------------------------------------------------------------------- forward

// R tokens per TPR threads, their rows' loads in flight together.
template <typename T, int N, int TPR, int R>
__global__ void __launch_bounds__(256) embedding_kernel(const __grid_constant__ EmbedArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int RPB = 256 / TPR;
  const int t = threadIdx.x % TPR;
  const int64_t first = ((int64_t)blockIdx.x * RPB + threadIdx.x / TPR) * R;
  using Pack = Vec<T, N>;
  const T* src[R];
  bool ok[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int64_t id = first + j < a.tokens ? id_at(a, first + j) : -1;
    ok[j] = id >= 0 && id < a.rows;
    src[j] = static_cast<const T*>(a.src) + (ok[j] ? id : 0) * a.ld_src;
  }
  for (int64_t c = (int64_t)t * N; c < a.width; c += TPR * N) {
    Pack p[R];
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (ok[j]) p[j] = *reinterpret_cast<const Pack*>(src[j] + c);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (first + j >= a.tokens) continue;
#pragma unroll
      for (int i = 0; i < N; ++i)
        p[j].v[i] = (T)(ok[j] ? to_f32<T>(p[j].v[i]) * a.scale : __int_as_float(0x7fffffff));
      *reinterpret_cast<Pack*>(static_cast<T*>(a.out) + (first + j) * a.ld_out + c) = p[j];
    }
  }
}

// ------------------------------------------------------------------------------- sorting

// The warps' counts of each digit, a row per digit (padded: the rows of 32 digits start on
// different banks).
template <int WARPS> struct DigitCounts {
  uint16_t n[kDigits][WARPS + 2];
  uint32_t scan[kDigits];
  uint32_t warps[32];
};

// Rank of this lane's digit among the equal ones of the warp's items so far, in order; `valid`
// lanes only.  The lanes with an equal digit are found bit by bit (eight ballots; a match
// instruction took several times as long).
template <int WARPS>
__device__ __forceinline__ uint32_t warp_rank(uint32_t digit, bool valid, DigitCounts<WARPS>& c) {
  uint32_t peers = __ballot_sync(0xffffffffu, valid);
#pragma unroll
  for (int b = 0; b < kBits; ++b) {
    const bool one = digit >> b & 1;
    const uint32_t ones = __ballot_sync(0xffffffffu, one);
    peers &= one ? ones : ~ones;
  }
  const uint32_t below = peers & ((1u << (threadIdx.x % 32)) - 1);
  uint16_t* at = &c.n[digit][threadIdx.x / 32];
  const uint32_t before = *at;
  __syncwarp();
  if (valid && below == 0) *at = (uint16_t)(before + __popc(peers));
  __syncwarp();
  return before + __popc(below);
}

// Turns the warps' digit counts into each warp's first position within the digit, and scan[d] into
// the digit's first position: after the smaller digits of the block, or base[d] (not null).  All
// threads, a power of two of warps.
template <int WARPS>
__device__ __forceinline__ void digit_starts(DigitCounts<WARPS>& c, const uint32_t* base) {
  __syncthreads();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int PER = 32 / WARPS;          // digits that a warp scans at once, WARPS lanes each
  for (int d0 = warp * (kDigits / WARPS); d0 < (warp + 1) * (kDigits / WARPS); d0 += PER) {
    const int d = d0 + lane / WARPS, w = lane % WARPS;
    const uint32_t v = c.n[d][w];
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < WARPS; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (w >= o) incl += up;
    }
    c.n[d][w] = (uint16_t)(incl - v);
    if (w == WARPS - 1) c.scan[d] = incl;
  }
  __syncthreads();
  if (base) {
    if (threadIdx.x < kDigits) c.scan[threadIdx.x] = base[threadIdx.x];
  } else if (warp < kDigits / 32) {        // exclusive scan over the digits
    const uint32_t v = c.scan[threadIdx.x];
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    c.scan[threadIdx.x] = incl - v;
    if (lane == 31) c.warps[warp] = incl;
  }
  __syncthreads();
  if (!base) {
    if (threadIdx.x < kDigits)
      for (int w = 0; w < warp; ++w) c.scan[threadIdx.x] += c.warps[w];
    __syncthreads();
  }
}

// start[v], end[v] from neighbouring keys.
__device__ __forceinline__ void mark_run(const EmbedArgs& a, int64_t i, uint32_t key, uint32_t before,
                                         uint32_t after) {
  if (key >= (uint32_t)a.rows) return;
  if (i == 0 || before != key) a.start[key] = (uint32_t)i;
  if (i == a.tokens - 1 || after != key) a.end[key] = (uint32_t)i + 1;
}

// Clears the table (unless the gradient is added to it) and the frequencies: block `block` of
// `blocks`, `threads` threads each.
__device__ __forceinline__ void clear_table(const EmbedArgs& a, int64_t block, int64_t blocks, int threads) {
  const int64_t first = block * threads + threadIdx.x, step = blocks * threads;
  if (!a.accumulate) {
    const int64_t n = a.rows * a.width;
    if (a.ld_out == a.width || a.rows == 1) {
      const int64_t head = min(n, (int64_t)((16 - (uintptr_t)a.dtable % 16) % 16 / 4));
      float4* body = reinterpret_cast<float4*>(a.dtable + head);
      const int64_t vecs = (n - head) / 4;
      for (int64_t i = first; i < vecs; i += step) body[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (first < head) a.dtable[first] = 0.f;
      if (first < n - head - vecs * 4) a.dtable[head + vecs * 4 + first] = 0.f;
    } else {
      for (int64_t row = block; row < a.rows; row += blocks)
        for (int64_t c = threadIdx.x; c < a.width; c += threads) a.dtable[row * a.ld_out + c] = 0.f;
    }
  }
  if (a.frequency)
    for (int64_t i = first; i < a.rows; i += step) a.frequency[i] = 0.f;
}
// Clears the rows that no token has, and their frequencies: kRestRows at a time by a warp.  A row v
// has tokens where the sorted keys have v at start[v]; the other rows' start is whatever the
// workspace held.
constexpr int kRestRows = 8;
template <int N> __device__ __forceinline__ void clear_rest(const EmbedArgs& a, int64_t block, int64_t blocks) {
  const int lane = threadIdx.x % 32, warps = blockDim.x / 32;
  for (int64_t r0 = (block * warps + threadIdx.x / 32) * kRestRows; r0 < a.rows;
       r0 += blocks * warps * kRestRows) {
    const int64_t row = r0 + lane;
    bool none = false;
    if (lane < kRestRows && row < a.rows) {
      const uint32_t at = __ldg(a.start + row);
      none = at >= a.tokens || __ldg(a.keys + at) != (uint32_t)row;
      if (none && a.frequency) a.frequency[row] = 0.f;
    }
    if (a.accumulate) continue;
    for (uint32_t todo = __ballot_sync(0xffffffffu, none); todo; todo &= todo - 1) {
      float* out = a.dtable + (r0 + __ffs(todo) - 1) * a.ld_out;
      if constexpr (N > 2) {
        for (int64_t c = lane * 4; c < a.width; c += 128)
          *reinterpret_cast<float4*>(out + c) = make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
        for (int64_t c = lane; c < a.width; c += 32) out[c] = 0.f;
      }
    }
  }
}
__global__ void __launch_bounds__(kSortThreads) clear_kernel(const __grid_constant__ EmbedArgs a) {
  pdl_wait();
  pdl_trigger();
  clear_table(a, blockIdx.x, gridDim.x, kSortThreads);
}

// Up to kSmallTokens tokens by the first cluster: block b holds items [b I, (b + 1) I) in every
// pass, its warp w 32 at a time from w I / 16 on.  What one block can hold (kAlone, 2048 tokens) one
// sorts without the barriers between blocks, 2 to 3 us sooner.  The other blocks clear the table.
struct SmallSort {
  uint32_t keys[kSmallTokens / kCluster];
  uint32_t vals[kSmallTokens / kCluster];
  DigitCounts<kSortThreads / 32> counts;
  uint32_t total[kDigits], base[kDigits];
};
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
template <bool kAlone>
__global__ void __cluster_dims__(kAlone ? 1 : kCluster, 1, 1) __launch_bounds__(kSortThreads)
    sort_small_kernel(const __grid_constant__ EmbedArgs a) {
  __shared__ SmallSort s;
  constexpr int ROUNDS = kSmallTokens / kCluster / kSortThreads;
  pdl_wait();
  pdl_trigger();
  constexpr int BLOCKS = kAlone ? 1 : kCluster;
  if (blockIdx.x >= BLOCKS) {
    clear_table(a, blockIdx.x - BLOCKS, gridDim.x - BLOCKS, kSortThreads);
    return;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank_in = kAlone ? 0 : tc::cluster_rank();
  const int n = (int)a.tokens;
  auto sync = [&]() {
    if (kAlone) __syncthreads();
    else tc::cluster_sync();
  };
  const int rounds = (n + BLOCKS * kSortThreads - 1) / (BLOCKS * kSortThreads);
  const int items = rounds * kSortThreads;          // of a block
  const int base_item = (int)rank_in * items;
  auto local = [&](int r) { return (warp * rounds + r) * 32 + lane; };
  uint32_t key[ROUNDS], val[ROUNDS], rank[ROUNDS];
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    if (r < rounds) {
      const int i = base_item + local(r);
      key[r] = i < n ? key_at(a, i) : 0;
      val[r] = (uint32_t)i;
    }
  }
  for (int pass = 0; pass < a.passes; ++pass) {
    for (int i = threadIdx.x; i < kDigits * (kSortThreads / 32 + 2); i += kSortThreads)
      s.counts.n[0][i] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r)
      if (r < rounds)
        rank[r] = warp_rank((key[r] >> (kBits * pass)) % kDigits, base_item + local(r) < n, s.counts);
    digit_starts(s.counts, nullptr);
    // every block's totals: the digits before this one, and this digit's in the blocks before
    const int d = threadIdx.x;
    if (d < kDigits)
      s.total[d] = (d + 1 < kDigits ? s.counts.scan[d + 1] : (uint32_t)max(0, min(items, n - base_item))) -
                   s.counts.scan[d];
    sync();
    uint32_t before = 0, all = 0;
    if (d < kDigits) {
      if (kAlone) {
        all = s.total[d];
      } else {
#pragma unroll
        for (uint32_t c = 0; c < kCluster; ++c) {
          const uint32_t v = ld_cluster_u32(tc::mapa(&s.total[d], c));
          before += c < rank_in ? v : 0;
          all += v;
        }
      }
      uint32_t incl = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      s.base[d] = incl - all + before;
      if (lane == 31) s.counts.warps[warp] = incl;
    }
    __syncthreads();
    if (d < kDigits)
      for (int w = 0; w < warp; ++w) s.base[d] += s.counts.warps[w];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      if (r < rounds && base_item + local(r) < n) {
        const uint32_t g = (key[r] >> (kBits * pass)) % kDigits;
        const uint32_t at = s.base[g] + s.counts.n[g][warp] + rank[r];
        if (kAlone) {
          s.keys[at] = key[r];
          s.vals[at] = val[r];
        } else {
          const uint32_t to = at / (uint32_t)items, off = at - to * (uint32_t)items;
          tc::st_cluster_u32(tc::mapa(&s.keys[off], to), key[r]);
          tc::st_cluster_u32(tc::mapa(&s.vals[off], to), val[r]);
        }
      }
    }
    sync();
    if (pass + 1 < a.passes) {
#pragma unroll
      for (int r = 0; r < ROUNDS; ++r) {
        if (r < rounds && base_item + local(r) < n) {
          key[r] = s.keys[local(r)];
          val[r] = s.vals[local(r)];
        }
      }
    }
  }
  for (int j = threadIdx.x; j < items && base_item + j < n; j += kSortThreads) {
    const int i = base_item + j;
    auto neighbour = [&](int k) -> uint32_t {      // the key at item k, of this block or the next one
      if (kAlone || k < 0 || k >= n) return 0;   // (one block's neighbours are its own)
      const int b = k / items;
      return ld_cluster_u32(tc::mapa(&s.keys[k - b * items], (uint32_t)b));
    };
    const uint32_t k = s.keys[j];
    a.keys[i] = k;
    a.vals[i] = s.vals[j];
    mark_run(a, i, k, j > 0 ? s.keys[j - 1] : neighbour(i - 1),
             j + 1 < items && i + 1 < n ? s.keys[j + 1] : neighbour(i + 1));
  }
  sync();   // no block's shared memory goes while another reads it
}

// A tile's counts of each digit.
__global__ void __launch_bounds__(kTileThreads) sort_hist_kernel(const __grid_constant__ EmbedArgs a,
                                                                 const uint32_t* keys, int pass) {
  __shared__ uint32_t counts[kDigits];
  pdl_wait();
  pdl_trigger();
  counts[threadIdx.x] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * kTileItems;
  for (int i = threadIdx.x; i < kTileItems && first + i < a.tokens; i += kTileThreads) {
    const uint32_t k = keys ? keys[first + i] : key_at(a, first + i);
    atomicAdd(&counts[(k >> (kBits * pass)) % kDigits], 1u);
  }
  __syncthreads();
  a.hist[(int64_t)threadIdx.x * a.tiles + blockIdx.x] = counts[threadIdx.x];
}
// Block d: exclusive scan of digit d's counts over the tiles, and their sum.
__global__ void __launch_bounds__(1024) sort_scan_kernel(const __grid_constant__ EmbedArgs a) {
  __shared__ uint32_t warps[32];
  pdl_wait();
  pdl_trigger();
  uint32_t* h = a.hist + (int64_t)blockIdx.x * a.tiles;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  uint32_t carry = 0;
  for (int first = 0; first < a.tiles; first += 1024) {
    const int i = first + threadIdx.x;
    const uint32_t v = i < a.tiles ? h[i] : 0;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += warps[w];
      all += warps[w];
    }
    if (i < a.tiles) h[i] = carry + before + incl - v;
    carry += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) a.total[blockIdx.x] = carry;
}
// A tile's items to their places.
__global__ void __launch_bounds__(kTileThreads)
    sort_scatter_kernel(const __grid_constant__ EmbedArgs a, const uint32_t* keys, const uint32_t* vals,
                        uint32_t* keys_out, uint32_t* vals_out, int pass) {
  constexpr int WARPS = kTileThreads / 32, ROUNDS = kTileItems / kTileThreads;
  __shared__ DigitCounts<WARPS> counts;
  __shared__ uint32_t base[kDigits];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < kDigits * (WARPS + 2); i += kTileThreads) counts.n[0][i] = 0;
  // digits before this one in the whole order, and this digit's items in the tiles before
  counts.scan[threadIdx.x] = a.total[threadIdx.x];
  __syncthreads();
  uint32_t before = 0;
  for (int d = 0; d < (int)threadIdx.x; ++d) before += counts.scan[d];
  base[threadIdx.x] = before + a.hist[(int64_t)threadIdx.x * a.tiles + blockIdx.x];
  __syncthreads();
  uint32_t key[ROUNDS], val[ROUNDS], rank[ROUNDS];
  const int64_t first = (int64_t)blockIdx.x * kTileItems + warp * ROUNDS * 32 + lane;
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int64_t i = first + r * 32;
    const bool valid = i < a.tokens;
    key[r] = !valid ? 0 : keys ? keys[i] : key_at(a, i);
    val[r] = !valid ? 0 : vals ? vals[i] : (uint32_t)i;
    rank[r] = warp_rank((key[r] >> (kBits * pass)) % kDigits, valid, counts);
  }
  digit_starts(counts, base);
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    if (first + r * 32 < a.tokens) {
      const uint32_t d = (key[r] >> (kBits * pass)) % kDigits;
      const uint32_t at = counts.scan[d] + counts.n[d][warp] + rank[r];
      keys_out[at] = key[r];
      vals_out[at] = val[r];
    }
  }
}
__global__ void __launch_bounds__(256) sort_runs_kernel(const __grid_constant__ EmbedArgs a) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.tokens) return;
  mark_run(a, i, a.keys[i], i > 0 ? a.keys[i - 1] : 0, i + 1 < a.tokens ? a.keys[i + 1] : 0);
}

// ------------------------------------------------------------------------------- summing

template <int N> __device__ __forceinline__ void load_floats(const float* p, float (&v)[N]) {
  if constexpr (N == 1) {
    v[0] = __ldcg(p);
  } else if constexpr (N == 2) {
    *reinterpret_cast<float2*>(&v[0]) = __ldcg(reinterpret_cast<const float2*>(p));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(&v[i]) = __ldcg(reinterpret_cast<const float4*>(p + i));
  }
}
template <int N> __device__ __forceinline__ void store_floats(float* p, const float (&v)[N]) {
  if constexpr (N == 1) {
    p[0] = v[0];
  } else if constexpr (N == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(p + i) = *reinterpret_cast<const float4*>(&v[i]);
  }
}
// A finished sum to its row's channels from c.
template <int N>
__device__ __forceinline__ void store_row(const EmbedArgs& a, uint32_t row, int64_t c, const float (&sum)[N]) {
  float* out = a.dtable + (int64_t)row * a.ld_out + c;
  float v[N];
  if (a.accumulate) load_floats<N>(out, v);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = a.accumulate ? fmaf(sum[i], a.scale, v[i]) : sum[i] * a.scale;
  store_floats<N>(out, v);
}

// A chunk of the sorted order per TPR threads: its tokens' rows are read whatever their ids, and
// summed run by run.  A run inside the chunk goes to its row; the part of one that crosses into the
// chunk before or behind goes to the workspace: slot 0 if the run began before the chunk, slot 1
// if it begins in it.  Each thread copies what it will add itself into slots of its own in shared
// memory, two stages of eight rows (cp.async; single bf16 elements by way of registers), so that
// sixteen rows are in flight and no barrier orders them; with the rows in registers the code for a
// run's end stood there eight times over, and the kernel took 40 us for 16384 x 2048 (bf16).
constexpr int kStageRows = 8;
template <typename T, int N, int TPR>
__global__ void __launch_bounds__(256) embedding_chunks_kernel(const __grid_constant__ EmbedArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  using Pack = Vec<T, N>;
  Pack* slots = reinterpret_cast<Pack*>(raw) + threadIdx.x;   // [2][kStageRows][256]
  pdl_wait();
  pdl_trigger();
  constexpr int RPB = 256 / TPR, R = kStageRows;
  const int t = threadIdx.x % TPR;
  const int64_t chunk = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const int64_t lo = chunk * a.chunk;
  if (lo >= a.tokens) return;
  const int64_t hi = min(lo + a.chunk, a.tokens);
  const uint32_t rows = (uint32_t)a.rows;
  const uint32_t before = lo > 0 ? __ldg(a.keys + lo - 1) : 0xffffffffu;   // (no key: see kMaxIds)
  const uint32_t after = hi < a.tokens ? __ldg(a.keys + hi) : 0xffffffffu;
  const int64_t c = ((int64_t)blockIdx.y * TPR + t) * N;
  const int lane = threadIdx.x % 32;
  if (c - lane * N >= a.width) return;   // a warp without columns
  const bool on = c < a.width;
  const T* src = static_cast<const T*>(a.src) + c;
  // the next 64 positions' keys and tokens, two per lane (of a warp all positions are the same): read one
  // by one where they are used they were a chain of loads (300 tokens of 2046 channels in bf16, 8000 rows:
  // 26 us for 34)
  uint32_t keys0, vals0, keys1, vals1;
  auto window = [&](int64_t at, uint32_t& k, uint32_t& v) {
    const bool in = at + lane < hi;
    k = in ? __ldg(a.keys + at + lane) : 0xffffffffu;
    v = in ? __ldg(a.vals + at + lane) : 0u;
  };
  window(lo, keys0, vals0);
  window(lo + 32, keys1, vals1);
  auto fetch = [&](int from, int stage) {   // position `from` of the windows
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int p = from + j;               // (R divides 32: a fetch lies in one window)
      const uint32_t k = __shfl_sync(0xffffffffu, from < 32 ? keys0 : keys1, p % 32);
      const uint32_t v = __shfl_sync(0xffffffffu, from < 32 ? vals0 : vals1, p % 32);
      if (on && k < rows) {
        const T* at = src + (int64_t)v * a.ld_src;
        Pack* to = slots + (stage * R + j) * 256;
        if constexpr (sizeof(Pack) == 16)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(to)), "l"(at) : "memory");
        else if constexpr (sizeof(Pack) == 8)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(tc::smem_u32(to)), "l"(at) : "memory");
        else if constexpr (sizeof(Pack) == 4)
          tc::cp_async4(to, at);
        else
          *to = *reinterpret_cast<const Pack*>(at);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float sum[N];
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = 0.f;
  uint32_t run = __shfl_sync(0xffffffffu, keys0, 0);
  int64_t begin = lo, base = lo;       // of the run in this chunk; of the windows
  fetch(0, 0);
  fetch(R, 1);
  int stage = 0;
  for (int64_t i = lo;;) {             // position i, the first behind the run included
    const uint32_t key = __shfl_sync(0xffffffffu, keys0, (int)(i - base));   // (none from hi on)
    if (key != run) {
      if (on && run < rows) {
        const bool from_before = begin == lo && before == run, goes_on = i == hi && after == run;
        if (from_before || goes_on) {
          store_floats<N>(a.part + (chunk * 2 + (from_before ? 0 : 1)) * a.width + c, sum);
        } else {
          store_row<N>(a, run, c, sum);
          if (c == 0 && a.frequency) a.frequency[run] = (float)(i - begin) * a.inv_tokens;
        }
      }
      if (i >= hi) break;
      run = key;
      begin = i;
#pragma unroll
      for (int k = 0; k < N; ++k) sum[k] = 0.f;
    }
    const int j = (int)(i - lo) % R;
    if (j == 0) asm volatile("cp.async.wait_group 1;" ::: "memory");
    if (on && run < rows) {
      const Pack p = slots[(stage * R + j) * 256];
#pragma unroll
      for (int k = 0; k < N; ++k) sum[k] += to_f32<T>(p.v[k]);
    }
    ++i;
    if (j == R - 1) {
      fetch((int)(i - base) + R, stage);   // the slots just read
      stage ^= 1;
      if (i - base == 32) {
        base = i;
        keys0 = keys1;
        vals0 = vals1;
        window(base + 32, keys1, vals1);
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The runs that cross chunks: a warp per border, which adds the parts if it is the first that the run
// crosses.  The parts of a run over more than kLong chunks (a hot id) are divided by the block's
// warps and added in order (by one warp, four at a time, the gradient of 13810 tokens of one id and
// 224 channels took 130 us, so 35; of 16384 of 2048 channels 186 and 92).  The blocks from `joins`
// on clear the rows without tokens.
constexpr int kLong = 32;
template <int N>
__global__ void __launch_bounds__(256) embedding_join_kernel(const __grid_constant__ EmbedArgs a, int joins) {
  __shared__ int is_long[8];
  __shared__ float sums[8][32 * N];
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x >= joins) {
    const int64_t each = gridDim.x - joins;
    clear_rest<N>(a, blockIdx.x - joins + blockIdx.y * each, each * gridDim.y);
    return;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t c = ((int64_t)blockIdx.y * 32 + lane) * N;
  const bool on = c < a.width;
  // adds parts [p0, p1) of the run that crosses into `chunk` first: 0 is slot 1 of the chunk before
  auto add = [&](int64_t chunk, int64_t p0, int64_t p1, float (&sum)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = 0.f;
    constexpr int AHEAD = 8;
    for (int64_t p = p0; p < p1; p += AHEAD) {
      float v[AHEAD][N];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (p + k < p1)
          load_floats<N>(a.part + (p + k == 0 ? chunk * 2 - 1 : (chunk + p + k - 1) * 2) * a.width + c, v[k]);
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (p + k < p1) {
#pragma unroll
          for (int i = 0; i < N; ++i) sum[i] += v[k][i];
        }
    }
  };
  auto parts_of = [&](int64_t chunk, uint32_t run) {
    return (int64_t)((__ldg(a.end + run) - 1) / (uint32_t)a.chunk) - chunk + 2;
  };
  const int64_t chunk = (int64_t)blockIdx.x * 8 + warp + 1, at = chunk * a.chunk;
  const uint32_t run = at < a.tokens ? __ldg(a.keys + at) : 0xffffffffu;
  bool first = run < (uint32_t)a.rows && __ldg(a.keys + at - 1) == run;
  int64_t parts = 0;
  if (first) {
    const uint32_t start = __ldg(a.start + run);
    first = (int64_t)start >= at - a.chunk;          // it crossed no border before
    parts = parts_of(chunk, run);
    if (first && lane == 0 && blockIdx.y == 0 && a.frequency)
      a.frequency[run] = (float)(__ldg(a.end + run) - start) * a.inv_tokens;
  }
  if (first && parts <= kLong && on) {
    float sum[N];
    add(chunk, 0, parts, sum);
    store_row<N>(a, run, c, sum);
  }
  if (lane == 0) is_long[warp] = first && parts > kLong;
  __syncthreads();
  for (int w = 0; w < 8; ++w) {
    if (!is_long[w]) continue;
    const int64_t from = (int64_t)blockIdx.x * 8 + w + 1;
    const uint32_t hot = __ldg(a.keys + from * a.chunk);
    const int64_t all = parts_of(from, hot), each = (all + 7) / 8;
    if (on) {
      float sum[N];
      add(from, min(all, warp * each), min(all, (warp + 1) * each), sum);
#pragma unroll
      for (int i = 0; i < N; ++i) sums[warp][lane * N + i] = sum[i];
    }
    __syncthreads();
    if (warp == 0 && on) {
      float sum[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        sum[i] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[i] += sums[k][lane * N + i];
      }
      store_row<N>(a, hot, c, sum);
    }
    __syncthreads();
  }
}

template <typename T, int N> void launch_forward(const EmbedArgs& a, cudaStream_t st) {
  const dim3 block(256);
  auto grid = [&](int per) { return dim3((unsigned)cdiv(a.tokens, per)); };
  // narrow rows: a warp each; several tokens per thread where there are tokens for every SM
  const bool many = a.tokens >= 16 * (int64_t)num_sms();
  if (cdiv(a.width, N) <= 64) {
    if (many) launch_pdl(embedding_kernel<T, N, 32, 4>, grid(32), block, 0, st, a);
    else launch_pdl(embedding_kernel<T, N, 32, 1>, grid(8), block, 0, st, a);
  } else {
    if (many) launch_pdl(embedding_kernel<T, N, 256, 4>, grid(4), block, 0, st, a);
    else launch_pdl(embedding_kernel<T, N, 256, 1>, grid(1), block, 0, st, a);
  }
}

template <typename T, int N, int TPR> kfac_status launch_sums_by(const EmbedArgs& a, cudaStream_t st) {
  const int64_t chunks = cdiv(a.tokens, a.chunk);
  constexpr size_t smem = 2 * kStageRows * 256 * N * sizeof(T);
  static OncePerDevice once;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !once(dev, [] {
        return cudaFuncSetAttribute(embedding_chunks_kernel<T, N, TPR>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess;
      })) {
    check_launch();   // keeps the runtime's message
    return KFAC_ERR_CUDA;
  }
  // (blocks of columns beside each other: 4096 tokens of 8191 channels, one block for all: 585 us)
  launch_pdl(embedding_chunks_kernel<T, N, TPR>,
             dim3((unsigned)cdiv(chunks, 256 / TPR), (unsigned)cdiv(a.width, TPR * N)), dim3(256), smem, st, a);
  constexpr int NJ = N < 4 ? N : 4;
  const unsigned columns = (unsigned)cdiv(a.width, 32 * NJ);
  const int joins = (int)cdiv(chunks - 1, 8);
  const int64_t rest = std::min<int64_t>(8 * (int64_t)num_sms(), cdiv(a.rows, 8 * kRestRows));
  const int clears = a.late ? (int)cdiv(rest, columns) : 0;
  if (joins + clears > 0)
    launch_pdl(embedding_join_kernel<NJ>, dim3((unsigned)(joins + clears), columns), dim3(256), 0, st, a, joins);
  return KFAC_OK;
}
template <typename T, int N> kfac_status launch_sums(const EmbedArgs& a, cudaStream_t st) {
  return cdiv(a.width, N) <= 64 ? launch_sums_by<T, N, 32>(a, st) : launch_sums_by<T, N, 256>(a, st);
}

// Sorted positions per chunk: at least two stages of rows, else one wave of the chunks' blocks (three
// per SM, of up to 2048 channels; narrow rows: eight chunks a block).  16384 x 2048 in bf16 in chunks
// of 36: sums and joins 25 and 7 us, of 16 (2.2 waves) 29 and 12.
int64_t chunks_of_wave(int64_t width) {
  const int64_t blocks = std::max<int64_t>(1, 3 * (int64_t)num_sms() / cdiv(std::max<int64_t>(width, 1), 2048));
  return width <= 512 ? 8 * blocks : blocks;
}
int chunk_of(int64_t tokens, int64_t width) {
  return (int)std::max<int64_t>(2 * kStageRows, cdiv(tokens, chunks_of_wave(width)));
}

struct Layout {
  size_t keys, vals, keys2, vals2, start, end, hist, total, part, bytes;
};
Layout layout_of(int64_t tokens, int64_t rows, int64_t width) {
  Layout l{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes);
    return here;
  };
  const bool small = tokens <= kSmallTokens;
  l.keys = take((size_t)tokens * 4);
  l.vals = take((size_t)tokens * 4);
  l.keys2 = take(small ? 0 : (size_t)tokens * 4);
  l.vals2 = take(small ? 0 : (size_t)tokens * 4);
  l.start = take((size_t)rows * 4);
  l.end = take((size_t)rows * 4);
  l.hist = take(small ? 0 : (size_t)cdiv(tokens, kTileItems) * kDigits * 4);
  l.total = take(small ? 0 : kDigits * 4);
  // as many parts as any smaller number of tokens takes: a chunk more than this one's can be fewer chunks
  const int64_t chunks = std::min(cdiv(tokens, 2 * kStageRows), chunks_of_wave(width));
  l.part = take(chunks > 1 ? (size_t)chunks * 2 * (size_t)width * 4 : 0);
  l.bytes = at;
  return l;
}

bool whole_vectors(const void* p, int64_t ld, int64_t rows, size_t es, int bytes) {
  return (uintptr_t)p % bytes == 0 && (rows == 1 || ld * (int64_t)es % bytes == 0);
}

kfac_status check_desc(const kfac_embedding_desc* d, size_t* es) {
  if (!d || (d->dtype != KFAC_F32 && d->dtype != KFAC_BF16)) return KFAC_ERR_INVALID_ARG;
  if ((d->id_bits != 32 && d->id_bits != 64) || d->tokens < 0 || d->rows < 0 || d->width < 0 ||
      !std::isfinite((float)d->scale))
    return KFAC_ERR_INVALID_ARG;
  if (d->tokens > kMaxIds || d->rows > kMaxIds || d->width > (int64_t(1) << 20))
    return KFAC_ERR_UNSUPPORTED;
  *es = d->dtype == KFAC_BF16 ? 2 : 4;
  return KFAC_OK;
}
bool bad_rows(const void* p, int64_t ld, int64_t rows, int64_t width, size_t es) {
  return !p || (uintptr_t)p % es || ld < 0 || ld > (int64_t(1) << 32) || (rows > 1 && ld < width);
}

}  // namespace
}  // namespace kfac

using namespace kfac;

extern "C" kfac_status kfac_embedding(const kfac_embedding_desc* d, const void* ids,
                                      const void* table, void* out, cudaStream_t stream) {
  size_t es = 0;
  if (kfac_status e = check_desc(d, &es)) return e;
  if (d->tokens == 0 || d->width == 0) return KFAC_OK;
  if (!ids || (uintptr_t)ids % (d->id_bits / 8) || bad_rows(out, d->ldo, d->tokens, d->width, es) ||
      (d->rows > 0 && bad_rows(table, d->ldt, d->rows, d->width, es)))
    return KFAC_ERR_INVALID_ARG;
  EmbedArgs a{};
  a.ids = ids;
  a.src = table;
  a.out = out;
  a.tokens = d->tokens;
  a.rows = d->rows;
  a.width = d->width;
  a.ld_src = d->ldt;
  a.ld_out = d->ldo;
  a.scale = (float)d->scale;
  a.id64 = d->id_bits == 64;
  // rows of whole vectors of n elements (16384 tokens of 2046 channels in bf16: pairs 23 us, elements 31)
  auto whole = [&](int n) {
    const int bytes = n * (int)es;
    return d->width % n == 0 && whole_vectors(table, d->ldt, d->rows, es, bytes) &&
           whole_vectors(out, d->ldo, d->tokens, es, bytes);
  };
  const bool vec = whole(16 / (int)es);
  if (d->dtype == KFAC_BF16) {
    if (vec) launch_forward<__nv_bfloat16, 8>(a, stream);
    else if (whole(2)) launch_forward<__nv_bfloat16, 2>(a, stream);
    else launch_forward<__nv_bfloat16, 1>(a, stream);
  } else {
    if (vec) launch_forward<float, 4>(a, stream);
    else if (whole(2)) launch_forward<float, 2>(a, stream);
    else launch_forward<float, 1>(a, stream);
  }
  count_launch();
  return check_launch();
}

extern "C" kfac_status kfac_embedding_workspace_size(int64_t tokens, int64_t rows, int64_t width,
                                                     size_t* bytes) {
  if (!bytes || tokens < 0 || rows < 0 || width < 0) return KFAC_ERR_INVALID_ARG;
  if (tokens > kMaxIds || rows > kMaxIds || width > (int64_t(1) << 20)) return KFAC_ERR_UNSUPPORTED;
  *bytes = layout_of(tokens, rows, width).bytes;
  return KFAC_OK;
}

extern "C" kfac_status kfac_embedding_backward(const kfac_embedding_desc* d, const void* ids,
                                               const void* dout, float* dtable, int64_t padding_id,
                                               int accumulate, float* frequency, void* workspace,
                                               size_t workspace_bytes, cudaStream_t stream) {
  size_t es = 0;
  if (kfac_status e = check_desc(d, &es)) return e;
  if ((accumulate != 0 && accumulate != 1) || padding_id < -1 || (uintptr_t)frequency % 4)
    return KFAC_ERR_INVALID_ARG;
  if (d->rows > 0 && d->width == 0 && frequency) return KFAC_ERR_INVALID_ARG;   // (no launch would write it)
  if (d->rows == 0 || d->width == 0) return KFAC_OK;
  if (bad_rows(dtable, d->ldt, d->rows, d->width, 4)) return KFAC_ERR_INVALID_ARG;
  if (d->tokens > 0 && (!ids || (uintptr_t)ids % (d->id_bits / 8) ||
                        bad_rows(dout, d->ldo, d->tokens, d->width, es)))
    return KFAC_ERR_INVALID_ARG;
  const Layout l = layout_of(d->tokens, d->rows, d->width);
  if (!workspace || (uintptr_t)workspace % kAlign || workspace_bytes < l.bytes) return KFAC_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  auto at = [&](size_t off) { return reinterpret_cast<uint32_t*>(ws + off); };
  EmbedArgs a{};
  a.ids = ids;
  a.src = dout;
  a.dtable = dtable;
  a.frequency = frequency;
  a.tokens = d->tokens;
  a.rows = d->rows;
  a.width = d->width;
  a.ld_src = d->ldo;
  a.ld_out = d->ldt;
  a.padding_id = padding_id;
  a.scale = (float)d->scale;
  a.inv_tokens = d->tokens ? (float)(1.0 / (double)d->tokens) : 0.f;
  a.id64 = d->id_bits == 64;
  a.accumulate = accumulate;
  for (a.passes = 1; a.passes < 4 && (d->rows >> (kBits * a.passes)) != 0;) ++a.passes;   // keys 0..rows
  a.keys = at(l.keys);
  a.vals = at(l.vals);
  a.keys2 = at(l.keys2);
  a.vals2 = at(l.vals2);
  a.start = at(l.start);
  a.end = at(l.end);
  a.hist = at(l.hist);
  a.total = at(l.total);
  a.tiles = (int)cdiv(d->tokens, kTileItems);
  a.part = reinterpret_cast<float*>(at(l.part));
  a.chunk = chunk_of(d->tokens, d->width);
  // Beside the one cluster's sort the table is cleared whole: the memory is idle then, and rows that the
  // sums write soon after are often still in L2 (16384 tokens, 50021 x 2048: 103 us, 108 with
  // only the first 50 to 160 MB cleared there and the rest behind the sums).  Where the sort is
  // launches of its own, only rows without tokens are, behind the sums (65536 tokens: 180 us for 225).
  a.late = d->tokens > kSmallTokens && (!accumulate || frequency);
  int launches = 0;
  // blocks that clear: a few per SM, or what there is to clear
  const int64_t clears =
      accumulate && !frequency
          ? 0
          : std::min<int64_t>(4 * (int64_t)num_sms(),
                              cdiv((accumulate ? 0 : cdiv(d->rows * d->width, 4)) + (frequency ? d->rows : 0),
                                   kSortThreads));
  if (d->tokens > 0 && d->tokens <= kSmallTokens) {
    if (d->tokens <= kSmallTokens / kCluster) {
      launch_pdl(sort_small_kernel<true>, dim3((unsigned)(1 + clears)), dim3(kSortThreads), 0, stream, a);
    } else {
      const dim3 grid((unsigned)(kCluster + cdiv(clears, kCluster) * kCluster));
      launch_pdl(sort_small_kernel<false>, grid, dim3(kSortThreads), 0, stream, a);
    }
    launches = 1;
  } else if (d->tokens == 0 && clears > 0) {
    launch_pdl(clear_kernel, dim3((unsigned)clears), dim3(kSortThreads), 0, stream, a);
    launches = 1;
  }
  if (d->tokens == 0) {
    count_launch(launches);
    return check_launch();
  }
  if (d->tokens > kSmallTokens) {
    // the last pass ends in keys, vals
    const uint32_t *k = nullptr, *v = nullptr;
    for (int pass = 0; pass < a.passes; ++pass) {
      const bool to_first = (a.passes - pass) % 2 == 1;
      uint32_t *ko = to_first ? a.keys : a.keys2, *vo = to_first ? a.vals : a.vals2;
      launch_pdl(sort_hist_kernel, dim3((unsigned)a.tiles), dim3(kTileThreads), 0, stream, a, k, pass);
      launch_pdl(sort_scan_kernel, dim3(kDigits), dim3(1024), 0, stream, a);
      launch_pdl(sort_scatter_kernel, dim3((unsigned)a.tiles), dim3(kTileThreads), 0, stream, a, k, v,
                 ko, vo, pass);
      k = ko;
      v = vo;
    }
    launch_pdl(sort_runs_kernel, dim3((unsigned)cdiv(d->tokens, 256)), dim3(256), 0, stream, a);
    launches += 3 * a.passes + 1;
  }
  // rows of whole vectors of n elements (16384 tokens of 2046 channels, 8000 rows: bf16 in pairs 74 us, in
  // elements 124, fp32 86 and 111)
  auto whole = [&](int n) {
    return d->width % n == 0 && whole_vectors(dout, d->ldo, d->tokens, es, n * (int)es) &&
           whole_vectors(dtable, d->ldt, d->rows, 4, std::min(4 * n, 16));
  };
  const bool vec = whole(16 / (int)es);
  const kfac_status e =
      d->dtype == KFAC_BF16
          ? (vec        ? launch_sums<__nv_bfloat16, 8>(a, stream)
             : whole(2) ? launch_sums<__nv_bfloat16, 2>(a, stream)
                        : launch_sums<__nv_bfloat16, 1>(a, stream))
          : (vec        ? launch_sums<float, 4>(a, stream)
             : whole(2) ? launch_sums<float, 2>(a, stream)
                        : launch_sums<float, 1>(a, stream));
  if (e) return e;
  count_launch(launches + 1 + (d->tokens > a.chunk));
  return check_launch();
}
