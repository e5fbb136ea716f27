// Rotary positions of query and key heads, and the table of cosines and sines.
//
//   pair i of a head at position t:  y0 = x0 c - x1 s,  y1 = x0 s + x1 c,
//   c = table[t][i], s = table[t][R/2 + i]; the inverse (the backward pass: the
//   rotation is orthogonal up to the table's scale) takes -s.  Half layout: pair i
//   is channels (i, i + R/2); interleaved: (2i, 2i + 1).  Channels from R on are
//   copied (nothing to do in place).
//
// Bound by memory: 3 flop per loaded element.  One launch serves q and k.  A thread
// keeps the cosines and sines of its VEC pairs in registers and applies them to
// kHeads = 2 heads of its token: four 16-byte loads in flight at 64 registers.  VEC
// is the widest vector (up to 16 bytes) that every address, stride and size allows.
// 16384 tokens, 16 + 16 heads of 128 bf16 (269 MB): 48 us, 5.6 TB/s.  Heads per thread,
// same case: 1: 52 us, 2: 49 us, 4: 66 us (registers leave too few blocks), 8: 101 us;
// 128 threads a block, not 256: 48 us.
// Arithmetic in fp32 whatever the type, one rounding at the store.
#include "kfac_internal.cuh"

#include <cmath>

namespace kfac {
namespace {

constexpr int kHeads = 2;        // heads per thread
constexpr int kRopeThreads = 128;

struct RopeArgs {
  const void* x[2];              // q, k
  void* y[2];
  int64_t xs[2][3], ys[2][3];    // strides (batch, row, head) in elements
  int heads[2];
  const float* table;
  int64_t table_rows;
  const int* positions;          // null: offset + row
  int64_t pos_stride;            // elements between the positions of two batch entries
  int64_t offset;
  int length, dim, rotary;
  float sign;                    // -1: inverse
  int chunks, rot_chunks;        // chunks of 2 VEC channels per head; those that rotate
  int groups;                    // head groups per token
  int64_t items;                 // batch * length * groups * chunks
};

template <typename T, int VEC> struct alignas(sizeof(T) * VEC) Vec { T v[VEC]; };

template <typename T, int VEC, bool kInter>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  pdl_wait();
  pdl_trigger();
  using V = Vec<T, VEC>;
  const int64_t item = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x;
  if (item >= a.items) return;
  // chunk fastest, then head group, then token (32-bit divisions: the host keeps
  // groups * chunks below 2^31 and the token in 64 bits)
  const uint32_t per_token = (uint32_t)a.groups * (uint32_t)a.chunks;
  const int64_t token = item < INT64_C(0x7fffffff) ? (int64_t)((uint32_t)item / per_token)
                                                   : item / per_token;
  const uint32_t rem = (uint32_t)(item - token * per_token);
  const int group = (int)(rem / (uint32_t)a.chunks), chunk = (int)(rem % (uint32_t)a.chunks);
  const int64_t b = token < INT64_C(0x7fffffff) ? (int64_t)((uint32_t)token / (uint32_t)a.length)
                                                : token / a.length;
  const int row = (int)(token - b * a.length);
  const bool rot = chunk < a.rot_chunks;
  const int half = a.rotary / 2;
  // channels of the chunk's two vectors
  int c0, c1;
  bool has1 = true;
  if (rot) {
    c0 = kInter ? 2 * VEC * chunk : VEC * chunk;
    c1 = kInter ? c0 + VEC : c0 + half;
  } else {
    c0 = a.rotary + 2 * VEC * (chunk - a.rot_chunks);
    c1 = c0 + VEC;
    has1 = c1 < a.dim;
  }
  const int total = a.heads[0] + a.heads[1];
  V in0[kHeads], in1[kHeads];
  T* out[kHeads];
  bool on[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const int h = group + j * a.groups;
    on[j] = h < total;
    out[j] = nullptr;
    if (!on[j]) continue;
    const int w = h < a.heads[0] ? 0 : 1;
    const int hh = w ? h - a.heads[0] : h;
    const T* x = static_cast<const T*>(a.x[w]) + b * a.xs[w][0] + row * a.xs[w][1] + hh * a.xs[w][2];
    out[j] = static_cast<T*>(a.y[w]) + b * a.ys[w][0] + row * a.ys[w][1] + hh * a.ys[w][2];
    if (!rot && out[j] == x) {   // in place: these channels stay
      on[j] = false;
      continue;
    }
    in0[j] = *reinterpret_cast<const V*>(x + c0);
    if (has1) in1[j] = *reinterpret_cast<const V*>(x + c1);
  }
  if (!rot) {
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      if (!on[j]) continue;
      *reinterpret_cast<V*>(out[j] + c0) = in0[j];
      if (has1) *reinterpret_cast<V*>(out[j] + c1) = in1[j];
    }
    return;
  }
  const int64_t pos = a.positions ? (int64_t)a.positions[b * a.pos_stride + row] : a.offset + row;
  float cs[VEC], sn[VEC];
  if (pos >= 0 && pos < a.table_rows) {
    constexpr int TV = VEC < 4 ? VEC : 4;   // 16-byte table loads where VEC covers them
    using TVec = Vec<float, TV>;
    const float* t = a.table + pos * a.rotary + VEC * chunk;
#pragma unroll
    for (int i = 0; i < VEC; i += TV) {
      const TVec c = *reinterpret_cast<const TVec*>(t + i), s = *reinterpret_cast<const TVec*>(t + half + i);
#pragma unroll
      for (int e = 0; e < TV; ++e) {
        cs[i + e] = c.v[e];
        sn[i + e] = s.v[e] * a.sign;
      }
    }
  } else {   // outside the table: no value to give
#pragma unroll
    for (int i = 0; i < VEC; ++i) cs[i] = sn[i] = __int_as_float(0x7fffffff);
  }
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    if (!on[j]) continue;
    V o0, o1;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float p, q;
      if (kInter) {
        p = to_f32<T>(2 * i < VEC ? in0[j].v[(2 * i) % VEC] : in1[j].v[(2 * i) % VEC]);
        q = to_f32<T>(2 * i + 1 < VEC ? in0[j].v[(2 * i + 1) % VEC] : in1[j].v[(2 * i + 1) % VEC]);
      } else {
        p = to_f32<T>(in0[j].v[i]);
        q = to_f32<T>(in1[j].v[i]);
      }
      const T y0 = (T)(p * cs[i] - q * sn[i]), y1 = (T)(p * sn[i] + q * cs[i]);
      if (kInter) {
        if (2 * i < VEC) o0.v[(2 * i) % VEC] = y0; else o1.v[(2 * i) % VEC] = y0;
        if (2 * i + 1 < VEC) o0.v[(2 * i + 1) % VEC] = y1; else o1.v[(2 * i + 1) % VEC] = y1;
      } else {
        o0.v[i] = y0;
        o1.v[i] = y1;
      }
    }
    *reinterpret_cast<V*>(out[j] + c0) = o0;
    *reinterpret_cast<V*>(out[j] + c1) = o1;
  }
}

// Angles in 64 bits: at position 10^6 an fp32 angle is off by 0.03 rad.  Bound by the 64-bit
// sines, cosines and powers (131072 rows x 128: 1.1 ms, YARN 1.4 ms; a table is made once).
struct RopeTableArgs {
  float* table;
  int64_t rows;
  int rotary;
  double log2_base;     // of the base after scaling
  int scaling;
  double factor;
  double low, high;     // YARN: pair index where the blend begins and ends
  double magnitude;
};

__global__ void __launch_bounds__(256) rope_table_kernel(const RopeTableArgs a) {
  pdl_wait();
  pdl_trigger();
  const int half = a.rotary / 2;
  const int64_t n = a.rows * half;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) {
    const int64_t t = e / half;
    const int i = (int)(e - t * half);
    double f = exp2(-a.log2_base * (2.0 * i / a.rotary));
    if (a.scaling == KFAC_ROPE_LINEAR) f /= a.factor;
    if (a.scaling == KFAC_ROPE_YARN) {
      const double r = fmin(fmax((i - a.low) / (a.high - a.low), 0.0), 1.0);
      f = f * (1.0 - r) + f / a.factor * r;
    }
    double s, c;
    sincos((double)t * f, &s, &c);
    a.table[t * a.rotary + i] = (float)(c * a.magnitude);
    a.table[t * a.rotary + half + i] = (float)(s * a.magnitude);
  }
}

template <typename T, int VEC>
void launch_vec(const RopeArgs& a, bool inter, cudaStream_t st) {
  const unsigned grid = (unsigned)cdiv(a.items, kRopeThreads);
  if (inter) launch_pdl(rope_kernel<T, VEC, true>, dim3(grid), dim3(kRopeThreads), 0, st, a);
  else launch_pdl(rope_kernel<T, VEC, false>, dim3(grid), dim3(kRopeThreads), 0, st, a);
}

// Whether every vector of `vec` elements a thread touches is whole and aligned.
bool vec_ok(const RopeArgs& a, int es, int vec, bool inter) {
  // vectors start at multiples of vec in each half (half layout) or in the rotated
  // part (interleaved, 2 vec per chunk), and at multiples of vec behind it
  if (a.rotary % (2 * vec) || a.dim % vec) return false;
  if ((uintptr_t)a.table % (sizeof(float) * (vec < 4 ? vec : 4))) return false;
  (void)inter;
  const size_t bytes = (size_t)es * vec;
  for (int w = 0; w < 2; ++w) {
    if (!a.heads[w]) continue;
    if ((uintptr_t)a.x[w] % bytes || (uintptr_t)a.y[w] % bytes) return false;
    for (int i = 0; i < 3; ++i)
      if (a.xs[w][i] % vec || a.ys[w][i] % vec) return false;
  }
  return true;
}

}  // namespace
}  // namespace kfac

using namespace kfac;

extern "C" {

kfac_status kfac_rope(const kfac_rope_desc* d, const void* q, const void* k, const float* table,
                      const int* positions, void* out_q, void* out_k, cudaStream_t stream) {
  if (!d || !table || (uintptr_t)table % sizeof(float)) return KFAC_ERR_INVALID_ARG;
  if (d->dtype != KFAC_F32 && d->dtype != KFAC_BF16) return KFAC_ERR_INVALID_ARG;
  if (d->interleaved != 0 && d->interleaved != 1) return KFAC_ERR_INVALID_ARG;
  if (d->inverse != 0 && d->inverse != 1) return KFAC_ERR_INVALID_ARG;
  if (d->batch < 0 || d->length < 0 || d->heads < 0 || d->kv_heads < 0) return KFAC_ERR_INVALID_ARG;
  if (d->head_dim < 1 || d->head_dim > 65536 || d->heads > 65536 || d->kv_heads > 65536)
    return KFAC_ERR_INVALID_ARG;
  if (d->rotary_dim < 2 || d->rotary_dim % 2 || d->rotary_dim > d->head_dim)
    return KFAC_ERR_INVALID_ARG;
  if (d->table_rows < 1 || d->position_offset < 0) return KFAC_ERR_INVALID_ARG;
  if (positions && (uintptr_t)positions % sizeof(int)) return KFAC_ERR_INVALID_ARG;
  if (!positions && d->position_offset > d->table_rows - d->length) return KFAC_ERR_INVALID_ARG;
  const int es = d->dtype == KFAC_BF16 ? 2 : 4;
  RopeArgs a{};
  a.x[0] = q;
  a.x[1] = k;
  a.y[0] = out_q;
  a.y[1] = out_k;
  a.heads[0] = d->heads;
  a.heads[1] = d->kv_heads;
  for (int i = 0; i < 3; ++i) {
    a.xs[0][i] = d->q_stride[i];
    a.xs[1][i] = d->k_stride[i];
    a.ys[0][i] = d->out_q_stride[i];
    a.ys[1][i] = d->out_k_stride[i];
  }
  for (int w = 0; w < 2; ++w) {
    if (!a.heads[w]) continue;
    if (!a.x[w] || !a.y[w] || (uintptr_t)a.x[w] % es || (uintptr_t)a.y[w] % es)
      return KFAC_ERR_INVALID_ARG;
    const int64_t n[3] = {d->batch, d->length, a.heads[w]};
    for (int i = 0; i < 3; ++i) {
      if (a.xs[w][i] < 0 || a.ys[w][i] < 0) return KFAC_ERR_INVALID_ARG;
      if (n[i] > 1 && a.ys[w][i] < d->head_dim) return KFAC_ERR_INVALID_ARG;   // rows would overlap
      if (a.x[w] == a.y[w] && n[i] > 1 && a.xs[w][i] != a.ys[w][i]) return KFAC_ERR_INVALID_ARG;
      if (n[i] <= 1) a.xs[w][i] = a.ys[w][i] = 0;   // never multiplied: no say in alignment
    }
  }
  if (d->batch == 0 || d->length == 0 || d->heads + d->kv_heads == 0) return KFAC_OK;
  a.table = table;
  a.table_rows = d->table_rows;
  a.positions = positions;
  a.pos_stride = d->position_stride;
  a.offset = d->position_offset;
  a.length = d->length;
  a.dim = d->head_dim;
  a.rotary = d->rotary_dim;
  a.sign = d->inverse ? -1.f : 1.f;
  const bool inter = d->interleaved != 0;
  int vec = 16 / es;
  while (vec > 1 && !vec_ok(a, es, vec, inter)) vec /= 2;
  a.rot_chunks = a.rotary / 2 / vec;
  a.chunks = a.rot_chunks + (int)cdiv(a.dim - a.rotary, 2 * vec);
  a.groups = (int)cdiv(d->heads + d->kv_heads, kHeads);
  a.items = (int64_t)d->batch * d->length * a.groups * a.chunks;
  if (cdiv(a.items, kRopeThreads) > INT32_MAX) return KFAC_ERR_INVALID_ARG;
  if (es == 2) {
    if (vec == 8) launch_vec<__nv_bfloat16, 8>(a, inter, stream);
    else if (vec == 4) launch_vec<__nv_bfloat16, 4>(a, inter, stream);
    else if (vec == 2) launch_vec<__nv_bfloat16, 2>(a, inter, stream);
    else launch_vec<__nv_bfloat16, 1>(a, inter, stream);
  } else {
    if (vec == 4) launch_vec<float, 4>(a, inter, stream);
    else if (vec == 2) launch_vec<float, 2>(a, inter, stream);
    else launch_vec<float, 1>(a, inter, stream);
  }
  count_launch();
  return check_launch();
}

kfac_status kfac_rope_table(float* table, int64_t rows, int rotary_dim, double base, int scaling,
                            double factor, double original_length, cudaStream_t stream) {
  if (!table || (uintptr_t)table % sizeof(float) || rows < 0 || rows > (int64_t(1) << 40) ||
      rotary_dim < 2 || rotary_dim % 2 || rotary_dim > 65536)
    return KFAC_ERR_INVALID_ARG;
  if (!std::isfinite(base) || base <= 1.0) return KFAC_ERR_INVALID_ARG;
  if (scaling < KFAC_ROPE_PLAIN || scaling > KFAC_ROPE_YARN) return KFAC_ERR_INVALID_ARG;
  if (scaling != KFAC_ROPE_PLAIN && (!std::isfinite(factor) || factor < 1.0))
    return KFAC_ERR_INVALID_ARG;
  if (scaling == KFAC_ROPE_YARN && (!std::isfinite(original_length) || original_length < 1.0))
    return KFAC_ERR_INVALID_ARG;
  if (scaling == KFAC_ROPE_NTK && rotary_dim < 4) return KFAC_ERR_INVALID_ARG;
  if (rows == 0) return KFAC_OK;
  RopeTableArgs a{};
  a.table = table;
  a.rows = rows;
  a.rotary = rotary_dim;
  a.log2_base = std::log2(base);
  a.scaling = scaling;
  a.factor = factor;
  a.magnitude = 1.0;
  if (scaling == KFAC_ROPE_NTK)
    a.log2_base += std::log2(factor) * rotary_dim / (rotary_dim - 2.0);
  if (scaling == KFAC_ROPE_YARN) {
    // (Peng, Quesnelle, Fan, Shippole, "YaRN: efficient context window extension of large
    // language models", 2023.)
    // pair i turns original_length f_i / 2 pi times within the original length; pairs
    // with 32 turns or more keep their frequency, those with one or less are
    // interpolated, a linear blend over the index between
    const double pi2 = 6.283185307179586;
    auto index_of = [&](double turns) {
      return rotary_dim * std::log2(original_length / (turns * pi2)) / (2.0 * a.log2_base);
    };
    a.low = std::fmax(std::floor(index_of(32.0)), 0.0);
    a.high = std::fmin(std::ceil(index_of(1.0)), rotary_dim - 1.0);
    if (a.high <= a.low) a.high = a.low + 0.001;
    a.magnitude = 0.1 * std::log(factor) + 1.0;
  }
  const int64_t blocks = cdiv(rows * (rotary_dim / 2), 256);
  const unsigned grid = (unsigned)(blocks < 16 * num_sms() ? blocks : 16 * num_sms());
  launch_pdl(rope_table_kernel, dim3(grid), dim3(256), 0, stream, a);
  count_launch();
  return check_launch();
}

}  // extern "C"
