// k_append.cu -- tp_qkv_append: per-head norms, rotation, and the write of the
// keys and values into the paged cache, in one pass over the fused QKV buffer.
//
// Per token t, rank r and head h, with x the head's D values:
//   y = x * rsqrt(mean(x^2) + eps) * g          (queries and keys, where g is given)
//   (a, b) -> (a cos - b sin, b cos + a sin)     (queries and keys, the first `rot` values)
// in float32, rounded once to the cache's type.  Queries go to q[r][t], keys and
// values to page slot / page, row slot % page.
//
// D/8 lanes hold one head, each two quarters of 4 values: a lane below rot/8
// values 4l.. and rot/2 + 4l.. (with neighbouring pairs 8l.. and 8l + 4..), so
// that a pair never leaves its lane and every lane of the rotation needs the
// cosines and sines 4l..; the lanes behind the rotation hold 8l.. and 8l + 4...
// Only the mean is summed over lanes.
//
// Bytes bound it: each value is read and written once.  Two forms:
//   append_kernel       a group of lanes takes one head of one token: as many
//                       groups as there are heads, for small calls and rows that
//                       8-byte copies cannot take;
//   append_ring_kernel  a group takes four heads of a token after the other, the
//                       next token's heads, cosines and sines on their way into
//                       shared memory meanwhile (each lane copies its own
//                       pieces, so nothing is shared and no barrier is needed).
// Measured: 16384 tokens of 8 ranks x 12 heads of 128, bfloat16, normed and turned,
// 162 us (5.0 TB/s, 74% of the copy rate); with every head loaded in one piece and
// the rotation's partners shuffled, 270; one head a group 356.  One token 2.0 us.
// The ring starts where every resident block has two rounds: with fewer the
// first form's blocks are all resident at once and its loads overlap as well.
#include "attn.cuh"
#include "mma16.cuh"
#include "ptx.cuh"

namespace tp {
namespace {

// Four consecutive values, one access where vec.
template <typename T>
__device__ __forceinline__ void load4(const T *p, bool vec, float *x) {
  if constexpr (sizeof(T) == 4) {
    if (vec) {
      const float4 v = __ldcs(reinterpret_cast<const float4 *>(p));
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
      return;
    }
  } else if (vec) {
    const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
    const float2 lo = Half2<T>::unpack(v.x), hi = Half2<T>::unpack(v.y);
    x[0] = lo.x, x[1] = lo.y, x[2] = hi.x, x[3] = hi.y;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = static_cast<float>(p[i]);
}
template <typename T>
__device__ __forceinline__ void store4(T *p, bool vec, const float *x) {
  const uint2 v = make_uint2(Half2<T>::pack(x[0], x[1]), Half2<T>::pack(x[2], x[3]));
  if (vec) {
    *reinterpret_cast<uint2 *>(p) = v;
  } else {
    uint16_t *h = reinterpret_cast<uint16_t *>(p);
    h[0] = (uint16_t)v.x, h[1] = (uint16_t)(v.x >> 16), h[2] = (uint16_t)v.y, h[3] = (uint16_t)(v.y >> 16);
  }
}
__device__ __forceinline__ void table4(const float *p, bool vec, float *x) {
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
  bool in, q, rope, gain;  // one access for four values possible
};

// A lane's place: where its two quarters of a head begin.
struct Lane {
  int id, o0, o1;
  bool turns;     // they are pairs to rotate
  uint32_t mask;  // the lanes of its group: groups of one warp may take different branches
};
template <int D>
__device__ __forceinline__ Lane lane_of(const AppendArgs &a) {
  constexpr int L = D / 8;
  Lane l;
  l.id = threadIdx.x % L;
  l.mask = ((1u << L) - 1) << (threadIdx.x % 32 - l.id);
  l.turns = l.id < a.rot / 8;
  const bool halves = l.turns && !a.interleaved;
  l.o0 = halves ? 4 * l.id : 8 * l.id;
  l.o1 = halves ? a.rot / 2 + 4 * l.id : 8 * l.id + 4;
  return l;
}

struct Slot {
  int64_t page;
  int row;  // -1: not written
};
__device__ __forceinline__ Slot slot_of(const AppendArgs &a, int64_t slot, const Lane &l) {
  if (slot >= a.pages << a.page_log2) {
    if (l.id == 0) record_bad_value(a.status);
    slot = -1;
  }
  return Slot{slot >> a.page_log2, slot < 0 ? -1 : (int)slot & (a.page - 1)};
}
// The lane's cosines at position pos; its sines are rot/2 behind.
__device__ __forceinline__ const float *factors_of(const AppendArgs &a, int64_t pos, const Lane &l) {
  if (pos < 0 || pos >= a.rope_rows) {
    if (l.id == 0) record_bad_value(a.status);
    pos = 0;
  }
  return a.rope + pos * a.rot + 4 * l.id;
}

// Norm, rotation and store of heads h0 .. h0 + NH - 1 of token t, step by step
// for all of them: one head's steps wait for each other.
template <typename T, int D, int NH>
__device__ __forceinline__ void put_heads(const AppendArgs &a, const Aligned &vec, const Lane &l, int r, int64_t t, int h0,
                                          const Slot &slot, const float (&c)[4], const float (&s)[4],
                                          float (&y)[NH][8]) {
  const int H = a.Hq + 2 * a.Hk, turned = a.Hq + a.Hk;
  if (h0 < turned && (a.q_norm || a.k_norm)) {
    float sum[NH];
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      sum[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[i] = fmaf(y[i][j], y[i][j], sum[i]);
    }
#pragma unroll
    for (int m = D / 16; m > 0; m /= 2)
#pragma unroll
      for (int i = 0; i < NH; ++i) sum[i] += __shfl_xor_sync(l.mask, sum[i], m);
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      const float *gains = h0 + i < a.Hq ? a.q_norm : h0 + i < turned ? a.k_norm : nullptr;
      if (gains) {
        float g[8];
        table4(gains + l.o0, vec.gain, g);
        table4(gains + l.o1, vec.gain, g + 4);
        const float inv = rsqrtf(sum[i] * (1.0f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[i][j] *= inv * g[j];
      }
    }
  }
  if (l.turns) {
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      if (h0 + i >= turned) continue;
      float (&v)[8] = y[i];
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = v[2 * j], q = v[2 * j + 1];
          v[2 * j] = p * c[j] - q * s[j], v[2 * j + 1] = q * c[j] + p * s[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = v[j], q = v[j + 4];
          v[j] = p * c[j] - q * s[j], v[j + 4] = q * c[j] + p * s[j];
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NH; ++i) {
    const int h = h0 + i;
    if (h >= H) break;
    if (h < a.Hq) {
      T *q = static_cast<T *>(a.q[r]) + t * a.ldq + (int64_t)h * D;
      store4<T>(q + l.o0, vec.q, y[i]);
      store4<T>(q + l.o1, vec.q, y[i] + 4);
    } else if (slot.row >= 0) {
      const int kh = h < turned ? h - a.Hq : h - turned;
      T *row = static_cast<T *>(h < turned ? a.k_cache[r] : a.v_cache[r]) + slot.page * a.ld_page +
               ((int64_t)kh * a.page + slot.row) * D;
      store4<T>(row + l.o0, true, y[i]);
      store4<T>(row + l.o1, true, y[i] + 4);
    }
  }
}

// Block (x, y, z): x tokens, y a head, z a rank.
template <typename TIn, typename T, int D>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a, const Aligned vec) {
  constexpr int L = D / 8;  // lanes of a head
  griddep_launch_dependents();
  griddep_wait();
  const Lane l = lane_of<D>(a);
  const int64_t t = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  if (t >= a.T) return;
  const int r = blockIdx.z, h = blockIdx.y;
  float x[1][8], c[4], s[4];
  const TIn *src = static_cast<const TIn *>(a.qkv[r]) + t * a.ld + (int64_t)h * D;
  load4<TIn>(src + l.o0, vec.in, x[0]);
  load4<TIn>(src + l.o1, vec.in, x[0] + 4);
  Slot slot{0, -1};
  if (h >= a.Hq) slot = slot_of(a, __ldg(a.slots + t), l);
  if (l.turns && h < a.Hq + a.Hk) {
    const float *f = factors_of(a, __ldg(a.positions + t), l);
    table4(f, vec.rope, c);
    table4(f + a.rot / 2, vec.rope, s);
  }
  put_heads<T, D, 1>(a, vec, l, r, t, h, slot, c, s, x);
}

template <typename TIn>
struct Ring {
  static constexpr int kHeads = 4, kStages = 2;
  static constexpr int kQuarter = 4 * sizeof(TIn);  // bytes
  static constexpr int kRope = kStages * kHeads * 2 * kQuarter * kThreads;  // where cosines and sines begin
  static constexpr int kSmem = kRope + kStages * 32 * kThreads;
};

// Block (x, y, z): token blocks x, x + gridDim.x, ..; y a stretch of four heads, z a rank.
template <typename TIn, typename T, int D>
__global__ void __launch_bounds__(kThreads, 3)
    append_ring_kernel(const __grid_constant__ AppendArgs a, const Aligned vec) {
  using R = Ring<TIn>;
  constexpr int L = D / 8, kTokens = kThreads / L, NH = R::kHeads;
  extern __shared__ __align__(16) uint8_t smem[];
  griddep_launch_dependents();
  griddep_wait();
  const Lane l = lane_of<D>(a);
  const int r = blockIdx.z, H = a.Hq + 2 * a.Hk, h0 = blockIdx.y * NH;
  const int64_t first = (int64_t)blockIdx.x * kTokens + threadIdx.x / L, step = (int64_t)gridDim.x * kTokens;
  const TIn *src = static_cast<const TIn *>(a.qkv[r]) + (int64_t)h0 * D;
  const bool turns = l.turns && h0 < a.Hq + a.Hk, keeps = h0 + NH > a.Hq;
  // a piece of one lane lies beside its neighbours': piece 2i, 2i + 1 head i's quarters
  auto at = [&](int stage, int piece) { return ((stage * NH * 2 + piece) * kThreads + (int)threadIdx.x) * R::kQuarter; };
  auto rope_at = [&](int stage, int piece) { return R::kRope + ((stage * 2 + piece) * kThreads + (int)threadIdx.x) * 16; };
  const uint32_t base = smem_u32(smem);

  int64_t ahead = first;  // the token to copy next
  int next_pos = turns && ahead < a.T ? __ldg(a.positions + ahead) : 0;
  auto copy = [&](int stage) {
    if (ahead < a.T) {
      const TIn *row = src + ahead * a.ld;
#pragma unroll
      for (int i = 0; i < NH; ++i)
        if (h0 + i < H) {
          cp_async<R::kQuarter>(base + at(stage, 2 * i), row + i * D + l.o0);
          cp_async<R::kQuarter>(base + at(stage, 2 * i + 1), row + i * D + l.o1);
        }
      if (turns) {
        const float *f = factors_of(a, next_pos, l);
        cp_async<16>(base + rope_at(stage, 0), f);
        cp_async<16>(base + rope_at(stage, 1), f + a.rot / 2);
      }
      ahead += step;
      if (turns && ahead < a.T) next_pos = __ldg(a.positions + ahead);
    }
    cp_async_commit();
  };
  auto read4 = [&](int at, float *x) {
    if constexpr (sizeof(TIn) == 4) {
      const float4 v = *reinterpret_cast<const float4 *>(smem + at);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2 *>(smem + at);
      const float2 lo = Half2<TIn>::unpack(v.x), hi = Half2<TIn>::unpack(v.y);
      x[0] = lo.x, x[1] = lo.y, x[2] = hi.x, x[3] = hi.y;
    }
  };
  copy(0);
  int stage = 0;
  for (int64_t t = first; t < a.T; t += step) {
    const int64_t at_slot = keeps ? __ldg(a.slots + t) : -1;
    copy(stage ^ 1);
    cp_async_wait<1>();
    float c[4], s[4], y[NH][8];
    if (turns) {
      const float4 fc = *reinterpret_cast<const float4 *>(smem + rope_at(stage, 0));
      const float4 fs = *reinterpret_cast<const float4 *>(smem + rope_at(stage, 1));
      c[0] = fc.x, c[1] = fc.y, c[2] = fc.z, c[3] = fc.w;
      s[0] = fs.x, s[1] = fs.y, s[2] = fs.z, s[3] = fs.w;
    }
#pragma unroll
    for (int i = 0; i < NH; ++i) read4(at(stage, 2 * i), y[i]), read4(at(stage, 2 * i + 1), y[i] + 4);
    Slot slot{0, -1};
    if (keeps) slot = slot_of(a, at_slot, l);
    put_heads<T, D, NH>(a, vec, l, r, t, h0, slot, c, s, y);
    stage ^= 1;
  }
  cp_async_wait<0>();
}

template <typename TIn, typename T, int D>
int launch(const AppendArgs &a, cudaStream_t s) {
  const int H = a.Hq + 2 * a.Hk;
  constexpr int kTokens = kThreads / (D / 8);
  auto aligned = [](const void *p, int bytes) { return (uintptr_t)p % bytes == 0; };
  constexpr int in_bytes = 4 * sizeof(TIn);
  Aligned vec;
  vec.in = (a.ld * (int64_t)sizeof(TIn)) % in_bytes == 0, vec.q = (a.ldq * 2) % 8 == 0;
  for (int r = 0; r < a.N; ++r) {
    vec.in = vec.in && aligned(a.qkv[r], in_bytes);
    vec.q = vec.q && aligned(a.q[r], 8);
  }
  vec.rope = aligned(a.rope, 16), vec.gain = aligned(a.q_norm, 16) && aligned(a.k_norm, 16);
  const int64_t blocks = (a.T + kTokens - 1) / kTokens;
  if (blocks > 0x7fffffff) return set_error(TP_ERR_UNSUPPORTED, "too many tokens for one launch");
  cudaError_t e;
  using R = Ring<TIn>;
  const int stretches = (H + R::kHeads - 1) / R::kHeads;
  const int64_t resident = (3 * sm_count() + stretches * a.N - 1) / (stretches * a.N);  // token blocks at a time
  if (vec.in && vec.rope && blocks >= 2 * resident) {
    auto kern = append_ring_kernel<TIn, T, D>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kSmem);
    if (e == cudaSuccess)
      e = launch_pdl(kern, dim3((unsigned)resident, (unsigned)stretches, (unsigned)a.N), dim3(kThreads), R::kSmem, s, a,
                     vec);
  } else {
    e = launch_pdl(append_kernel<TIn, T, D>, dim3((unsigned)blocks, (unsigned)H, (unsigned)a.N), dim3(kThreads), 0, s, a,
                   vec);
  }
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
