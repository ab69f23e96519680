// attn.cuh -- what the attention-side kernels share: the arguments of the
// append, the two paged attentions and the token draw, and small device helpers.
//
// The paged cache of one rank is (pages, Hk, page, D): a page holds `page`
// consecutive positions of one sequence, and within a page each key-value
// head's positions lie side by side, so 16 positions of a head are one
// contiguous block.  `ld_page` is the distance in elements between pages
// (Hk * page * D, or more when keys and values share an allocation).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tp_internal.h"

namespace tp {

// Positions of a sequence and rows of q at most: sums of two of them, a tile's
// end and a window's beginning stay inside 32 bits.
constexpr int64_t kMostPositions = 1 << 30;

struct AppendArgs {
  const void *qkv[kMaxShards];
  void *q[kMaxShards], *k_cache[kMaxShards], *v_cache[kMaxShards];
  const float *q_norm, *k_norm;  // nullable, (D)
  const float *rope;             // nullable, (rope_rows, rot): cosines, then sines
  const int32_t *positions;      // (T), read where rope is given
  const int64_t *slots;          // (T)
  int64_t T, ld, ldq, pages, ld_page, rope_rows;
  int N, Hq, Hk, D, page, page_log2, rot, interleaved;
  int in_dt, dt;
  float eps;
  int *status;
};

struct AttnArgs {
  const void *q[kMaxShards], *k_cache[kMaxShards], *v_cache[kMaxShards];
  void *o[kMaxShards];
  const int32_t *block_table;  // (B, width), row stride ld_table
  const int32_t *seq_lens;     // (B)
  const int32_t *cu_seqlens;   // (B + 1), or null: one query token per sequence
  const int32_t *prefix_lens;  // nullable, (B)
  int64_t T, B, ldq, ldo, pages, ld_page, ld_table, width;
  int64_t cap;                 // positions that a row of the table holds, kMostPositions at most
  int N, Hq, Hk, D, page, page_log2;
  int dt, window;              // window 0: none
  float scale, softcap;        // softcap 0: none
  int *status;
};

struct SampleArgs {
  const void *logits;
  const float *u, *temperature, *top_p, *min_p;  // all but u nullable
  const int32_t *top_k;                          // nullable
  int64_t *tokens;
  float *logprobs;  // nullable
  int64_t B, V, ld;
  int in_dt;
};

int launch_append(const AppendArgs &a, cudaStream_t s);
int launch_decode(const AttnArgs &a, cudaStream_t s);
int launch_prefill(const AttnArgs &a, cudaStream_t s);
int launch_attn_simt(const AttnArgs &a, cudaStream_t s);
int launch_sample(const SampleArgs &a, cudaStream_t s);

#ifdef __CUDACC__

template <typename T>
struct Half2;  // packed pairs of the 16-bit types
template <>
struct Half2<__nv_bfloat16> {
  typedef __nv_bfloat162 Pair;
  static constexpr bool kBf16 = true;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&v);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
};
template <>
struct Half2<__half> {
  typedef __half2 Pair;
  static constexpr bool kBf16 = false;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&v);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return __half22float2(*reinterpret_cast<__half2 *>(&u));
  }
};

// Records a bad value found in device memory (a page, slot or position out of
// range), which tp_query_status() reports.  The kernel goes on to its end.
__device__ __forceinline__ void record_bad_value(int *status) { atomicCAS(status, 0, TP_ERR_INVALID_ARG); }

#endif  // __CUDACC__

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// cap * tanh(z), given x = z * 2 log2(e): 1 - 2 / (1 + e^2z), and below |z| = 0.1, where
// that cancels (a cap of 10^6 would move scores by 0.1), tanh's series.  Both are within
// 5 parts in 10^6 of the score, less than half of a term's rounding to 16 bits for scores
// up to 50.
__device__ __forceinline__ float capped(float x, float cap) {
  const float z = x * 0.34657359f, z2 = z * z;
  const float wide = fmaf(-2.0f * cap, rcp_approx(1.0f + exp2_approx(x)), cap);
  const float series = cap * z * fmaf(z2, fmaf(z2, 0.13333333f, -0.33333333f), 1.0f);
  return fabsf(z) < 0.1f ? series : wide;
}

}  // namespace tp
