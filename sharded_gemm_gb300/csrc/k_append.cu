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

constexpr int kThreads = 256;

template <typename TIn, typename T, int D, int HPG>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a, int chunks,
                                                          int64_t groups, int vec_in, int vec_q) {
  constexpr int L = D / 8;  // lanes of a head
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x % L;
  // the lanes of this thread's group: groups of one warp may take different branches
  const uint32_t mask = ((1u << L) - 1) << (threadIdx.x % 32 - lane);
  const int64_t g = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / L;
  if (g >= groups) return;
  const int chunk = (int)(g % chunks);
  const int64_t unit = g / chunks;
  const int64_t t = unit % a.T;
  const int r = (int)(unit / a.T);
  const int H = a.Hq + 2 * a.Hk, h0 = chunk * HPG;
  const TIn *src = static_cast<const TIn *>(a.qkv[r]) + t * a.ld + lane * 8;

  float x[HPG][8];
#pragma unroll
  for (int i = 0; i < HPG; ++i)
    if (h0 + i < H) load8<TIn>(src + (int64_t)(h0 + i) * D, vec_in, x[i]);

  const int64_t slot = a.slots[t];
  bool write_kv = slot >= 0;
  if (slot >= a.pages * a.page) {
    write_kv = false;
    if (lane == 0) record_bad_value(a.status);
  }
  const int64_t pg = write_kv ? slot / a.page : 0;
  const int off = write_kv ? (int)(slot - pg * a.page) : 0;

  // Rotation: this lane's factors.  Halves: value i < rot/2 pairs with
  // i + rot/2, factor i.  Neighbours: values 2i, 2i + 1, factor i.
  const int half = a.rot / 2, i0 = lane * 8;
  const bool turns = i0 < a.rot;
  float c[8], s[8];
  if (turns && h0 < a.Hq + a.Hk) {
    int64_t pos = a.positions[t];
    if (pos < 0 || pos >= a.rope_rows) {
      pos = 0;
      if (lane == 0) record_bad_value(a.status);
    }
    const float *row = a.rope + pos * a.rot;
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[2 * i] = c[2 * i + 1] = __ldg(row + i0 / 2 + i);
        s[2 * i + 1] = __ldg(row + half + i0 / 2 + i);
        s[2 * i] = -s[2 * i + 1];
      }
    } else {
      const int f0 = i0 < half ? i0 : i0 - half;
      const float sign = i0 < half ? -1.0f : 1.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = __ldg(row + f0 + i);
        s[i] = sign * __ldg(row + half + f0 + i);
      }
    }
  }

#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    const int h = h0 + i;
    if (h >= H) break;
    float (&y)[8] = x[i];
    if (h < a.Hq + a.Hk) {
      const float *gain = h < a.Hq ? a.q_norm : a.k_norm;
      if (gain) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(y[j], y[j], sum);
#pragma unroll
        for (int m = L / 2; m > 0; m /= 2) sum += __shfl_xor_sync(mask, sum, m);
        const float inv = rsqrtf(sum * (1.0f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= inv * __ldg(gain + i0 + j);
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
        store8<T>(static_cast<T *>(a.q[r]) + t * a.ldq + (int64_t)h * D + i0, vec_q, y);
        continue;
      }
    }
    if (write_kv) {
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
  bool vec_in = (a.ld * (int64_t)sizeof(TIn)) % 16 == 0, vec_q = (a.ldq * 2) % 16 == 0;
  for (int r = 0; r < a.N; ++r) {
    vec_in = vec_in && (uintptr_t)a.qkv[r] % 16 == 0;
    vec_q = vec_q && (uintptr_t)a.q[r] % 16 == 0;
  }
  const bool wide = a.T * a.N * H >= 8192;
  const int hpg = wide ? 4 : 1;
  const int chunks = (H + hpg - 1) / hpg;
  const int64_t groups = a.T * a.N * chunks;
  const int64_t blocks = (groups * (D / 8) + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return set_error(TP_ERR_UNSUPPORTED, "T * N * heads too large for one launch");
  const cudaError_t e =
      wide ? launch_pdl(append_kernel<TIn, T, D, 4>, dim3((unsigned)blocks), dim3(kThreads), 0, s, a, chunks, groups,
                        (int)vec_in, (int)vec_q)
           : launch_pdl(append_kernel<TIn, T, D, 1>, dim3((unsigned)blocks), dim3(kThreads), 0, s, a, chunks, groups,
                        (int)vec_in, (int)vec_q);
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
