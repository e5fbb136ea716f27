// Token embedding and its gradient by sorted tokens:
//   out[t] = scale table[ids[t]];   dtable[v] = scale sum_{t: ids[t] = v} dout[t].
//
// Both are bound by memory: the forward pass reads and writes a row per token, the gradient
// reads dout once and writes the whole table (the larger part for a large vocabulary).
// The gradient needs the tokens of each row together.  They are sorted by id with a stable
// radix sort (8 bits a pass, ranks from warp matches), so that every row is summed in the order
// of its tokens: no atomics, the same inputs give the same bits.  Up to 16384 tokens one block
// sorts in shared memory; beyond that, histogram, scan and scatter launches per pass.
// A row's run in the sorted order is found through start[v], which only rows with tokens have:
// start[v] counts only if the sorted key there is v and the one before it is not, so that the
// array needs no clearing.
// Text has hot ids (padding, articles): runs longer than a chunk of the sorted order are summed
// chunk by chunk first, by blocks of their own, and their row adds the chunks' sums in order.
#include "kfac_internal.cuh"
#include "per_device.h"

#include <algorithm>
#include <cmath>

namespace kfac {
namespace {

constexpr int64_t kMaxIds = (int64_t(1) << 31) - 2;
constexpr int kSmallTokens = 16384;    // sorted by one block
constexpr int kSortThreads = 1024;
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

// Rank of this lane's digit among the equal ones of the warp's items so far, in order:
// counts[d] is the warp's count of digit d before these 32 items and after them, `valid` lanes
// only.
__device__ __forceinline__ uint32_t warp_rank(uint32_t digit, bool valid, uint16_t* counts) {
  const uint32_t peers = __match_any_sync(0xffffffffu, valid ? digit : 0xffffffffu);
  const uint32_t below = peers & ((1u << (threadIdx.x % 32)) - 1);
  const uint32_t before = valid ? counts[digit] : 0;
  __syncwarp();
  if (valid && below == 0) counts[digit] = (uint16_t)(before + __popc(peers));
  __syncwarp();
  return before + __popc(below);
}

// Turns the warps' digit counts into each warp's first position of each digit, counted from the
// digits before it in the block; `base` (or null) is added per digit.  Threads >= kDigits.
template <int WARPS>
__device__ __forceinline__ void digit_starts(uint16_t (*counts)[kDigits], uint32_t* scan,
                                             const uint32_t* base) {
  __syncthreads();
  const int d = threadIdx.x;
  uint32_t mine = 0;
  if (d < kDigits)
    for (int w = 0; w < WARPS; ++w) mine += counts[w][d];
  // exclusive scan over the digits
  if (d < kDigits) scan[d] = mine;
  __syncthreads();
  if (d < 32) {
    uint32_t v[kDigits / 32], sum = 0;
#pragma unroll
    for (int i = 0; i < kDigits / 32; ++i) {
      v[i] = sum;
      sum += scan[d * (kDigits / 32) + i];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (d >= o) incl += up;
    }
#pragma unroll
    for (int i = 0; i < kDigits / 32; ++i) scan[d * (kDigits / 32) + i] = v[i] + incl - sum;
  }
  __syncthreads();
  if (d < kDigits) {
    if (base) scan[d] = base[d];
    uint32_t at = 0;
    for (int w = 0; w < WARPS; ++w) {   // within the digit
      const uint32_t n = counts[w][d];
      counts[w][d] = (uint16_t)at;
      at += n;
    }
  }
  __syncthreads();
}

// start[v], end[v] from neighbouring keys.
__device__ __forceinline__ void mark_run(const EmbedArgs& a, int64_t i, uint32_t key, uint32_t before,
                                         uint32_t after) {
  if (key >= (uint32_t)a.rows) return;
  if (i == 0 || before != key) a.start[key] = (uint32_t)i;
  if (i == a.tokens - 1 || after != key) a.end[key] = (uint32_t)i + 1;
}

// Up to kSmallTokens tokens.  Warp w takes items [w I, (w + 1) I) of every pass, 32 at a time.
struct SmallSort {
  uint32_t keys[kSmallTokens];
  uint32_t vals[kSmallTokens];
  uint16_t counts[kSortThreads / 32][kDigits];
  uint32_t scan[kDigits];
};
__global__ void __launch_bounds__(kSortThreads) sort_small_kernel(const __grid_constant__ EmbedArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  SmallSort& s = *reinterpret_cast<SmallSort*>(raw);
  constexpr int WARPS = kSortThreads / 32, ROUNDS = kSmallTokens / kSortThreads;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int n = (int)a.tokens;
  const int rounds = (int)((n + kSortThreads - 1) / kSortThreads);
  pdl_wait();
  pdl_trigger();
  uint32_t key[ROUNDS], val[ROUNDS], rank[ROUNDS];
  auto item = [&](int r) { return (warp * rounds + r) * 32 + lane; };
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    if (r < rounds) {
      const int i = item(r);
      key[r] = i < n ? key_at(a, i) : 0;
      val[r] = (uint32_t)i;
    }
  }
  for (int pass = 0; pass < a.passes; ++pass) {
    for (int i = threadIdx.x; i < WARPS * kDigits; i += kSortThreads) s.counts[0][i] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r)
      if (r < rounds)
        rank[r] = warp_rank((key[r] >> (kBits * pass)) % kDigits, item(r) < n, s.counts[warp]);
    digit_starts<WARPS>(s.counts, s.scan, nullptr);
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      if (r < rounds && item(r) < n) {
        const uint32_t d = (key[r] >> (kBits * pass)) % kDigits;
        const uint32_t at = s.scan[d] + s.counts[warp][d] + rank[r];
        s.keys[at] = key[r];
        s.vals[at] = val[r];
      }
    }
    __syncthreads();
    if (pass + 1 < a.passes) {
#pragma unroll
      for (int r = 0; r < ROUNDS; ++r) {
        if (r < rounds && item(r) < n) {
          key[r] = s.keys[item(r)];
          val[r] = s.vals[item(r)];
        }
      }
    }
  }
  for (int i = threadIdx.x; i < n; i += kSortThreads) {
    const uint32_t k = s.keys[i];
    a.keys[i] = k;
    a.vals[i] = s.vals[i];
    mark_run(a, i, k, i > 0 ? s.keys[i - 1] : 0, i + 1 < n ? s.keys[i + 1] : 0);
  }
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
  __shared__ uint16_t counts[WARPS][kDigits];
  __shared__ uint32_t scan[kDigits], base[kDigits];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < WARPS * kDigits; i += kTileThreads) counts[0][i] = 0;
  // digits before this one in the whole order, and this digit's items in the tiles before
  scan[threadIdx.x] = a.total[threadIdx.x];
  __syncthreads();
  uint32_t before = 0;
  for (int d = 0; d < (int)threadIdx.x; ++d) before += scan[d];
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
    rank[r] = warp_rank((key[r] >> (kBits * pass)) % kDigits, valid, counts[warp]);
  }
  digit_starts<WARPS>(counts, scan, base);
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    if (first + r * 32 < a.tokens) {
      const uint32_t d = (key[r] >> (kBits * pass)) % kDigits;
      const uint32_t at = scan[d] + counts[warp][d] + rank[r];
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

template <typename T, int N> struct Sum {
  float v[N];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
  }
  __device__ __forceinline__ void add(const Vec<T, N>& p) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += to_f32<T>(p.v[i]);
  }
};

// dout rows of sorted positions [lo, hi), channels from c, in order.
template <typename T, int N>
__device__ __forceinline__ void sum_rows(const EmbedArgs& a, uint32_t lo, uint32_t hi, int64_t c,
                                         Sum<T, N>& s) {
  const T* src = static_cast<const T*>(a.src) + c;
  uint32_t i = lo;
  for (; i + 4 <= hi; i += 4) {
    Vec<T, N> p[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      p[j] = *reinterpret_cast<const Vec<T, N>*>(src + (int64_t)__ldg(a.vals + i + j) * a.ld_src);
#pragma unroll
    for (int j = 0; j < 4; ++j) s.add(p[j]);
  }
  for (; i < hi; ++i)
    s.add(*reinterpret_cast<const Vec<T, N>*>(src + (int64_t)__ldg(a.vals + i) * a.ld_src));
}

// A chunk's share of the runs longer than a chunk: slot 0 of the one that covers its first
// position, slot 1 of one that begins behind it and covers its last.
template <typename T, int N, int TPR>
__global__ void __launch_bounds__(256) embedding_chunks_kernel(const __grid_constant__ EmbedArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int RPB = 256 / TPR;
  const int t = threadIdx.x % TPR;
  const int64_t chunk = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const int64_t lo = chunk * a.chunk;
  if (lo >= a.tokens) return;
  const int64_t hi = min(lo + a.chunk, a.tokens);
#pragma unroll
  for (int slot = 0; slot < 2; ++slot) {
    const uint32_t key = __ldg(a.keys + (slot ? hi - 1 : lo));
    if (key >= (uint32_t)a.rows) continue;
    const uint32_t start = __ldg(a.start + key), end = __ldg(a.end + key);
    if (end - start <= (uint32_t)a.chunk || (slot && start <= (uint32_t)lo)) continue;
    const uint32_t from = max(start, (uint32_t)lo), to = min(end, (uint32_t)hi);
    for (int64_t c = (int64_t)t * N; c < a.width; c += TPR * N) {
      Sum<T, N> s;
      s.clear();
      sum_rows<T, N>(a, from, to, c, s);
      float* p = a.part + (chunk * 2 + slot) * a.width + c;
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] = s.v[i];
    }
  }
}

// A row of the table per TPR threads.
template <typename T, int N, int TPR>
__global__ void __launch_bounds__(256) embedding_rows_kernel(const __grid_constant__ EmbedArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int RPB = 256 / TPR;
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (row >= a.rows) return;
  uint32_t start = a.start[row], end = 0;
  // whatever stands in start[row] where the row has no tokens, the keys do not agree with it
  if ((int64_t)start < a.tokens && a.keys[start] == (uint32_t)row &&
      (start == 0 || a.keys[start - 1] != (uint32_t)row))
    end = a.end[row];
  else
    start = 0;
  const uint32_t count = end - start;
  if (t == 0 && a.frequency) a.frequency[row] = (float)count * a.inv_tokens;
  if (count == 0 && a.accumulate) return;
  const uint32_t c0 = start / (uint32_t)a.chunk, c1 = count ? (end - 1) / (uint32_t)a.chunk : 0;
  for (int64_t c = (int64_t)t * N; c < a.width; c += TPR * N) {
    Sum<T, N> s;
    s.clear();
    if (count <= (uint32_t)a.chunk) {
      sum_rows<T, N>(a, start, end, c, s);
    } else {
      for (uint32_t k = c0; k <= c1; ++k) {
        const int slot = k == c0 && start != c0 * (uint32_t)a.chunk;
        const float* p = a.part + ((int64_t)k * 2 + slot) * a.width + c;
#pragma unroll
        for (int i = 0; i < N; ++i) s.v[i] += p[i];
      }
    }
    float* out = a.dtable + row * a.ld_out + c;
    if constexpr (N > 1) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        float4 o = make_float4(s.v[i] * a.scale, s.v[i + 1] * a.scale, s.v[i + 2] * a.scale,
                               s.v[i + 3] * a.scale);
        if (a.accumulate) {
          const float4 old = *reinterpret_cast<const float4*>(out + i);
          o = make_float4(o.x + old.x, o.y + old.y, o.z + old.z, o.w + old.w);
        }
        *reinterpret_cast<float4*>(out + i) = o;
      }
    } else {
      out[0] = s.v[0] * a.scale + (a.accumulate ? out[0] : 0.f);
    }
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

template <typename T, int N> void launch_sums(const EmbedArgs& a, cudaStream_t st) {
  const dim3 block(256);
  const int64_t chunks = cdiv(a.tokens, a.chunk);
  if (cdiv(a.width, N) <= 64) {
    if (a.tokens > a.chunk)
      launch_pdl(embedding_chunks_kernel<T, N, 32>, dim3((unsigned)cdiv(chunks, 8)), block, 0, st, a);
    launch_pdl(embedding_rows_kernel<T, N, 32>, dim3((unsigned)cdiv(a.rows, 8)), block, 0, st, a);
  } else {
    if (a.tokens > a.chunk)
      launch_pdl(embedding_chunks_kernel<T, N, 256>, dim3((unsigned)chunks), block, 0, st, a);
    launch_pdl(embedding_rows_kernel<T, N, 256>, dim3((unsigned)a.rows), block, 0, st, a);
  }
}

// Sorted positions per chunk: few enough that a row of one hot run adds few of them.
int chunk_of(int64_t tokens) {
  int c = 64;
  while (cdiv(tokens, c) > 4096) c *= 2;
  return c;
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
  const int chunk = chunk_of(tokens);
  l.part = take(tokens > chunk ? (size_t)cdiv(tokens, chunk) * 2 * (size_t)width * 4 : 0);
  l.bytes = at;
  return l;
}

bool whole_vectors(const void* p, int64_t ld, int64_t rows, size_t es) {
  return (uintptr_t)p % 16 == 0 && (rows == 1 || ld * (int64_t)es % 16 == 0);
}

kfac_status check_desc(const kfac_embedding_desc* d, size_t* es) {
  if (!d || (d->dtype != KFAC_F32 && d->dtype != KFAC_BF16)) return KFAC_ERR_INVALID_ARG;
  if ((d->id_bits != 32 && d->id_bits != 64) || d->tokens < 0 || d->rows < 0 || d->width < 0 ||
      !std::isfinite(d->scale))
    return KFAC_ERR_INVALID_ARG;
  if (d->tokens > kMaxIds || d->rows > kMaxIds || d->width > (int64_t(1) << 24))
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
  const int n = 16 / (int)es;
  const bool vec = d->width % n == 0 && whole_vectors(table, d->ldt, d->rows, es) &&
                   whole_vectors(out, d->ldo, d->tokens, es);
  if (d->dtype == KFAC_BF16) {
    if (vec) launch_forward<__nv_bfloat16, 8>(a, stream);
    else launch_forward<__nv_bfloat16, 1>(a, stream);
  } else {
    if (vec) launch_forward<float, 4>(a, stream);
    else launch_forward<float, 1>(a, stream);
  }
  count_launch();
  return check_launch();
}

extern "C" kfac_status kfac_embedding_workspace_size(int64_t tokens, int64_t rows, int64_t width,
                                                     size_t* bytes) {
  if (!bytes || tokens < 0 || rows < 0 || width < 0) return KFAC_ERR_INVALID_ARG;
  if (tokens > kMaxIds || rows > kMaxIds || width > (int64_t(1) << 24)) return KFAC_ERR_UNSUPPORTED;
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
  a.chunk = chunk_of(d->tokens);
  int launches = 0;
  if (d->tokens > 0 && d->tokens <= kSmallTokens) {
    static OncePerDevice once;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || !once(dev, [] {
          return cudaFuncSetAttribute(sort_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      (int)sizeof(SmallSort)) == cudaSuccess;
        })) {
      check_launch();
      return KFAC_ERR_CUDA;
    }
    launch_pdl(sort_small_kernel, dim3(1), dim3(kSortThreads), sizeof(SmallSort), stream, a);
    launches = 1;
  } else if (d->tokens > 0) {
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
    launches = 3 * a.passes + 1;
  }
  const int n = 16 / (int)es;
  const bool vec = d->width % n == 0 && (d->tokens == 0 || whole_vectors(dout, d->ldo, d->tokens, es)) &&
                   whole_vectors(dtable, d->ldt, d->rows, 4);
  if (d->dtype == KFAC_BF16) {
    if (vec) launch_sums<__nv_bfloat16, 8>(a, stream);
    else launch_sums<__nv_bfloat16, 1>(a, stream);
  } else {
    if (vec) launch_sums<float, 4>(a, stream);
    else launch_sums<float, 1>(a, stream);
  }
  count_launch(launches + 1 + (d->tokens > a.chunk));
  return check_launch();
}
