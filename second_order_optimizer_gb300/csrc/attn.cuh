// Shared by the cross-attention translation units.
#pragma once
#include "kfac_internal.cuh"
#include "per_device.h"

namespace kfac {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// One call's tensors.  Strides are (batch, row, head) in elements.  rows = group *
// len_q: the query rows that read one key head, query head (r / len_q) of the group
// and query r % len_q for row r.
struct Args {
  const void *q, *k, *v, *o, *dout;
  void *out, *dq, *dk, *dv;
  float* lse;                       // forward: written when not null
  const float* lse_in;              // backward
  float* delta;                     // backward: [batch][heads][len_q]
  const int* kv_len;
  const uint8_t* key_mask;
  int64_t qs[3], ks[3], vs[3], os[3], dos[3], dqs[3], dks[3], dvs[3];
  int batch, len_q, len_kv, heads, kv_heads, group, dim, rows;
  float scale;
  bool vec;                         // CUDA-core kernels: rows of whole 16-byte pieces
  int splits;                       // parts of the key axis (1: outputs written directly)
  int part_keys;                    // token kernel, more parts than a cluster: keys per part
  bool longest_first;               // token kernel: order of the batch entries
  float* part_o;                    // [splits][batch][kv_heads][rows][dim], normalised
  float* part_lse;                  // [splits][batch][kv_heads][rows]
  // backward: parts of the query rows for dK and dV, of the keys for dQ (1: outputs
  // written directly), and their fp32 sums, unscaled
  int dkv_splits, dq_splits;
  float *part_dk, *part_dv;         // [dkv_splits][batch][kv_heads][len_kv][dim]
  float* part_dq;                   // [dq_splits][batch][kv_heads][rows][dim]
};

// Permitted keys of batch entry b end here.
__device__ __forceinline__ int key_count(const Args& a, int b) {
  return a.kv_len ? min(max(__ldg(a.kv_len + b), 0), a.len_kv) : a.len_kv;
}
__device__ __forceinline__ bool key_ok(const Args& a, int b, int len, int key) {
  return key < len && (!a.key_mask || __ldg(a.key_mask + (int64_t)b * a.len_kv + key) != 0);
}
// Where a walk along the keys of batch entry b may end: behind the last permitted one (a
// mask that pads, or leaves nothing, then costs no tiles).  Whole warps; the search runs
// from the end, 512 keys at a time, and mostly ends with the first of them.
__device__ __forceinline__ int walk_end(const Args& a, int b) {
  const int len = key_count(a, b);
  if (!a.key_mask) return len;
  for (int key0 = (len - 1) / 512 * 512; key0 >= 0 && len > 0; key0 -= 512) {
    int last = -1;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int key = key0 + 32 * i + (int)(threadIdx.x % 32);
      if (key_ok(a, b, len, key)) last = key;
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (last >= 0) return last + 1;
  }
  return 0;
}
// Whether batch entry b has exactly one permitted key.  Its softmax is the constant 1 then,
// and dQ and dK are exactly zero, where P (dP - delta) would leave the rounding of its
// terms.  Whole warps; ends at the second key found.
__device__ __forceinline__ bool one_key(const Args& a, int b, int len) {
  if (!a.key_mask) return len == 1;
  int n = 0;
  for (int key0 = 0; key0 < len && n < 2; key0 += 512) {
    int mine = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) mine += key_ok(a, b, len, key0 + 32 * i + (int)(threadIdx.x % 32));
    n += __reduce_add_sync(0xffffffffu, mine);
  }
  return n == 1;
}
// Offset of packed row r of key head hk.
__device__ __forceinline__ int64_t row_offset(const Args& a, const int64_t (&s)[3], int b, int hk,
                                              int r) {
  const int g = r / a.len_q, i = r - g * a.len_q;
  return b * s[0] + i * s[1] + (int64_t)(hk * a.group + g) * s[2];
}

// Lets a kernel's blocks have this much dynamic shared memory on the current device.
template <typename K> kfac_status allow_smem(OncePerDevice& once, K kern, size_t bytes) {
  int dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && once(dev, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) ==
               cudaSuccess;
      }))
    return KFAC_OK;
  check_launch();   // keeps the runtime's message
  return KFAC_ERR_CUDA;
}

// Few query rows (bf16, rows that tc_forward_ok accepts).
constexpr int kTokenWarps = 4;
constexpr int kTokenPerSm = 3;      // resident blocks per SM
constexpr int kTokenCluster = 8;    // parts that one cluster joins
constexpr int kTokenOrdered = 32 * kTokenWarps;   // batch entries that it can order
kfac_status token_forward(const Args& a, cudaStream_t st);
// delta from P dP, of batch entries with at most kExactKeys permitted keys alone (bf16, the
// tensors of tc_backward_ok).
constexpr int kExactKeys = 128;
kfac_status delta_keys(const Args& a, cudaStream_t st);

// fp32 arithmetic: forward and backward (a.delta already written).
template <typename T> kfac_status f32_forward(const Args& a, cudaStream_t st);
template <typename T> kfac_status f32_backward(const Args& a, cudaStream_t st);
// The same for the bf16 tensors that the fp32 kernels take.
kfac_status f32_delta(const Args& a, cudaStream_t st);

// Tensor-core kernels (bf16): whether these tensors can take them, and their launches.
bool tc_forward_ok(const Args& a);
kfac_status tc_forward(const Args& a, cudaStream_t st);
int tc_forward_tiles(int dim, int len_q, int len_kv);   // of 128 queries per block: 1 or 2
bool tc_backward_ok(const Args& a);
kfac_status tc_backward(const Args& a, cudaStream_t st);   // a.delta already written

}  // namespace attn
}  // namespace kfac
