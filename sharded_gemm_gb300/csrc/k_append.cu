// k_append.cu -- tp_qkv_append: per-head norms, rotation, and the write of the
// keys and values into the paged cache, in one pass over the fused QKV buffer.
//
// Per token t, rank r and head h, with x the head's D values:
//   y = x * rsqrt(mean(x^2) + eps) * g          (queries and keys, where g is given)
//   (a, b) -> (a cos - b sin, b cos + a sin)     (queries and keys, the first `rot` values)
// in float32, rounded once to the cache's type.  Queries go to q[r][t], keys and
// values to page slot / page, row slot % page.
//
// D/8 lanes hold one head, eight values (16 bytes of a 16-bit type) each, so the
// mean is a few shuffles and the rotation's partner (rot/2 values away) sits in
// another lane of the group at the same place.  A group takes HPG heads of one
// token: their loads are issued together, and the token's cosines and sines are
// read once for all of them.  Bytes bound it: each value is read and written once.
#include "attn.cuh"
#include "ptx.cuh"

namespace tp {
namespace {

template <typename T>
__device__ __forceinline__ void load8(const T *p, bool vec, float (&x)[8]);

template <>
__device__ __forceinline__ void load8<float>(const float *p, bool vec, float (&x)[8]) {
  if (vec) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = p[i];
  }
}

template <typename T>
__device__ __forceinline__ void load8_16(const T *p, bool vec, float (&x)[8]) {
  if (vec) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Half2<T>::unpack(w[i]);
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(p[i]);
  }
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, bool vec, float (&x)[8]) {
  load8_16(p, vec, x);
}
template <>
__device__ __forceinline__ void load8<__half>(const __half *p, bool vec, float (&x)[8]) {
  load8_16(p, vec, x);
}

template <typename T>
__device__ __forceinline__ void store8(T *p, bool vec, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = Half2<T>::pack(x[2 * i], x[2 * i + 1]);
  if (vec) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    uint16_t *h = reinterpret_cast<uint16_t *>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[2 * i] = (uint16_t)w[i], h[2 * i + 1] = (uint16_t)(w[i] >> 16);
  }
}

// 8 consecutive floats of a table, 16-byte aligned where vec.
__device__ __forceinline__ void table8(const float *p, bool vec, float (&x)[8]) {
  if (vec) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __ldg(p + i);
  }
}
__device__ __forceinline__ void table4(const float *p, bool vec, float (&x)[4]) {
  if (vec) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __ldg(p + i);
  }
}

constexpr int kThreads = 256;

struct Aligned {
  bool in, q, rope, gain;  // 16-byte accesses possible
};

// Block (x, y, z): x tokens, y a stretch of HPG heads, z a rank.
template <typename TIn, typename T, int D, int HPG>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a, const Aligned vec) {
  constexpr int L = D / 8;  // lanes of a head
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x % L;
  // the lanes of this thread's group: groups of one warp may take different branches
  const uint32_t mask = ((1u << L) - 1) << (threadIdx.x % 32 - lane);
  const int64_t t = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  if (t >= a.T) return;
  const int r = blockIdx.z, H = a.Hq + 2 * a.Hk, h0 = blockIdx.y * HPG, i0 = lane * 8;
  const TIn *src = static_cast<const TIn *>(a.qkv[r]) + t * a.ld + i0;

  float x[HPG][8];
#pragma unroll
  for (int i = 0; i < HPG; ++i)
    if (h0 + i < H) load8<TIn>(src + (int64_t)(h0 + i) * D, vec.in, x[i]);

  int64_t slot = -1;
  if (h0 + HPG > a.Hq) {
    slot = __ldg(a.slots + t);
    if (slot >= a.pages << a.page_log2) {
      slot = -1;
      if (lane == 0) record_bad_value(a.status);
    }
  }
  const int64_t pg = slot >> a.page_log2;
  const int off = (int)slot & (a.page - 1);

  // Rotation: this lane's factors.  Halves: value i < rot/2 pairs with
  // i + rot/2, factor i.  Neighbours: values 2i, 2i + 1, factor i.
  const int half = a.rot / 2;
  const bool turns = i0 < a.rot;
  float c[8], s[8];
  if (turns && h0 < a.Hq + a.Hk) {
    int64_t pos = __ldg(a.positions + t);
    if (pos < 0 || pos >= a.rope_rows) {
      pos = 0;
      if (lane == 0) record_bad_value(a.status);
    }
    const float *row = a.rope + pos * a.rot;
    if (a.interleaved) {
      float c4[4], s4[4];
      table4(row + i0 / 2, vec.rope, c4);
      table4(row + half + i0 / 2, vec.rope, s4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[2 * i] = c[2 * i + 1] = c4[i];
        s[2 * i] = -s4[i], s[2 * i + 1] = s4[i];
      }
    } else {
      const int f0 = i0 < half ? i0 : i0 - half;
      table8(row + f0, vec.rope, c);
      table8(row + half + f0, vec.rope, s);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = i0 < half ? -s[i] : s[i];
    }
  }

  float gain[8];
  const float *gain_of = nullptr;  // whose gains are held
#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    const int h = h0 + i;
    if (h >= H) break;
    float (&y)[8] = x[i];
    if (h < a.Hq + a.Hk) {
      const float *want = h < a.Hq ? a.q_norm : a.k_norm;
      if (want) {
        if (want != gain_of) table8(want + i0, vec.gain, gain);
        gain_of = want;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(y[j], y[j], sum);
#pragma unroll
        for (int m = L / 2; m > 0; m /= 2) sum += __shfl_xor_sync(mask, sum, m);
        const float inv = rsqrtf(sum * (1.0f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= inv * gain[j];
      }
      if (a.rot) {
        float p[8];
        if (a.interleaved) {
#pragma unroll
          for (int j = 0; j < 8; ++j) p[j] = y[j ^ 1];
        } else {
          const int step = half / 8;  // the partner's distance in lanes
          const int from = (lane < step ? lane + step : lane - step) & (L - 1);
#pragma unroll
          for (int j = 0; j < 8; ++j) p[j] = __shfl_sync(mask, y[j], from, L);
        }
        if (turns) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = fmaf(p[j], s[j], y[j] * c[j]);
        }
      }
      if (h < a.Hq) {
        store8<T>(static_cast<T *>(a.q[r]) + t * a.ldq + (int64_t)h * D + i0, vec.q, y);
        continue;
      }
    }
    if (slot >= 0) {
      const bool is_k = h < a.Hq + a.Hk;
      const int kh = h - a.Hq - (is_k ? 0 : a.Hk);
      T *page = static_cast<T *>(is_k ? a.k_cache[r] : a.v_cache[r]) + pg * a.ld_page;
      store8<T>(page + ((int64_t)kh * a.page + off) * D + i0, true, y);
    }
  }
}

template <typename TIn, typename T, int D>
int launch(const AppendArgs &a, cudaStream_t s) {
  const int H = a.Hq + 2 * a.Hk;
  auto aligned = [](const void *p) { return (uintptr_t)p % 16 == 0; };
  Aligned vec;
  vec.in = (a.ld * (int64_t)sizeof(TIn)) % 16 == 0, vec.q = (a.ldq * 2) % 16 == 0;
  for (int r = 0; r < a.N; ++r) {
    vec.in = vec.in && aligned(a.qkv[r]);
    vec.q = vec.q && aligned(a.q[r]);
  }
  vec.rope = aligned(a.rope), vec.gain = aligned(a.q_norm) && aligned(a.k_norm);
  const bool wide = a.T * a.N * H >= 8192;  // fewer: one head a group, for more groups
  const int hpg = wide ? 4 : 1;
  const int64_t blocks = (a.T + kThreads / (D / 8) - 1) / (kThreads / (D / 8)), stretches = (H + hpg - 1) / hpg;
  if (blocks > 0x7fffffff || stretches > 65535)
    return set_error(TP_ERR_UNSUPPORTED, "too many tokens or heads for one launch");
  const dim3 grid((unsigned)blocks, (unsigned)stretches, (unsigned)a.N), block(kThreads);
  const cudaError_t e = wide ? launch_pdl(append_kernel<TIn, T, D, 4>, grid, block, 0, s, a, vec)
                             : launch_pdl(append_kernel<TIn, T, D, 1>, grid, block, 0, s, a, vec);
  if (e != cudaSuccess) return cuda_error(e, "append launch");
  note_launch();
  return TP_OK;
}

template <typename TIn>
int launch_in(const AppendArgs &a, cudaStream_t s) {
  if (a.dt == TP_BF16)
    return a.D == 64 ? launch<TIn, __nv_bfloat16, 64>(a, s) : launch<TIn, __nv_bfloat16, 128>(a, s);
  return a.D == 64 ? launch<TIn, __half, 64>(a, s) : launch<TIn, __half, 128>(a, s);
}

}  // namespace

int launch_append(const AppendArgs &a, cudaStream_t s) {
  if (a.in_dt == TP_F32) return launch_in<float>(a, s);
  return a.in_dt == TP_BF16 ? launch_in<__nv_bfloat16>(a, s) : launch_in<__half>(a, s);
}

}  // namespace tp
