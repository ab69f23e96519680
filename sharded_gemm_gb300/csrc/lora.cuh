// lora.cuh -- what the adapters' kernels share: a call's tiles out of its plan, h as sums
// of 16-bit numbers, the loads of fragments.
//
// A warp-level m16n8k16 product takes its fragments straight from memory, 16 bytes a lane,
// because a contraction may go through its index in any order that both operands share: a
// quad's four lanes hold 8 neighbouring elements each, which feed two products (with R of
// 16 four, for one).  32 output columns are dealt to four products so that a lane ends with
// 16 bytes of neighbouring ones (b_row): of 16-bit outputs 8, of float32 ones twice 4, so
// that a quad's 16-byte accesses lie side by side.
#pragma once

#include <type_traits>

#include "mma16.cuh"
#include "serve.cuh"

namespace tp {

int launch_lora_prompt(const LoraArgs &a, int RP, cudaStream_t s);

namespace {

constexpr int kWarps = 8, kLoraThreads = kWarps * 32;

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// Four columns of h from `col` on.  Those behind the rank are 0 whatever the row: the zeros that
// stand for the adapter's missing rows make NaN of an infinite x, which would go on to all outputs.
__device__ __forceinline__ float4 scaled_h(const float4 &v, float scale, int col, int R) {
  return make_float4(col < R ? v.x * scale : 0.0f, col + 1 < R ? v.y * scale : 0.0f, col + 2 < R ? v.z * scale : 0.0f,
                     col + 3 < R ? v.w * scale : 0.0f);
}

// Two values as sums of N 16-bit numbers each.  A finite value stays one (bfloat16's
// rounding may pass its largest), and behind an infinite one come zeros, not NaN.
template <typename T, int N>
__device__ __forceinline__ void terms_of(float a, float b, uint32_t *to, int step) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t t = Half2<T>::pack(a, b);
    float2 h = Half2<T>::unpack(t);
    if (isinf(h.x) || isinf(h.y)) {
      if (Half2<T>::kBf16) {  // cut instead
        if (isinf(h.x) && !isinf(a)) t = (t & 0xffff0000u) | __float_as_uint(a) >> 16;
        if (isinf(h.y) && !isinf(b)) t = (t & 0xffffu) | (__float_as_uint(b) & 0xffff0000u);
        h = Half2<T>::unpack(t);
      }
      a = isinf(h.x) ? 0.0f : a - h.x, b = isinf(h.y) ? 0.0f : b - h.y;
    } else {
      a -= h.x, b -= h.y;
    }
    to[i * step] = t;
  }
}

// The tiles of `rows` tokens of a group; none where the tokens without an adapter are
// left alone.
__device__ __forceinline__ int tiles_of(const LoraArgs &a, const int4 &g, int rows, bool none) {
  if (g.x < 0 && !none) return 0;
  if (g.x >= a.n || g.y < 0 || g.z < 0 || (int64_t)g.y + g.z > a.T) {  // not a plan of this call
    record_bad_value(a.status);
    return 0;
  }
  return (g.z + rows - 1) / rows;
}
// (Read whether or not there are so many groups: the load need not wait for their number.)
__device__ __forceinline__ int4 group_at(const LoraArgs &a, int i, int groups) {
  int4 g = make_int4(-1, 0, 0, 0);
  if (i < a.most) g = __ldg(reinterpret_cast<const int4 *>(a.plan + 4) + i);
  return i < groups ? g : make_int4(-1, 0, 0, 0);
}

// Tile `tile` of the plan, counting on from group `base` (tiles `before` it): its adapter,
// first place and tokens; false behind the last.  The same in all lanes.
__device__ __forceinline__ bool find_tile(const LoraArgs &a, int groups, int rows, bool none, int64_t tile, int &base,
                                          int64_t &before, int4 &found) {
  const int lane = threadIdx.x % 32;
  for (; base < groups; base += 32) {
    const int4 g = group_at(a, base + lane, groups);
    const int mine = tiles_of(a, g, rows, none);
    int run = mine;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
      const int o = __shfl_up_sync(0xffffffffu, run, m);
      if (lane >= m) run += o;
    }
    const int all = __shfl_sync(0xffffffffu, run, 31);
    if (tile < before + all) {
      const int at = (int)(tile - before);
      const uint32_t in = __ballot_sync(0xffffffffu, at >= run - mine && at < run);
      const int l = __ffs(in) - 1, skip = (at - __shfl_sync(0xffffffffu, run - mine, l)) * rows;
      found.x = __shfl_sync(0xffffffffu, g.x, l);
      found.y = __shfl_sync(0xffffffffu, g.y, l) + skip;
      found.z = min(rows, __shfl_sync(0xffffffffu, g.z, l) - skip);
      return true;
    }
    before += all;
  }
  return false;
}

// The exponent that takes the largest finite value of a row of h to 2^14..2^15, below float16's
// largest (at most 126: its power's reciprocal is a normal number); the same in all lanes.
template <int RP>
__device__ __forceinline__ int row_exponent(const float *row) {
  float most = 0.0f;
  for (int c = threadIdx.x % 32; c < RP; c += 32) {
    const float v = fabsf(row[c]);
    most = fmaxf(most, v <= 3.402823466e38f ? v : 0.0f);
  }
  most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
  return most > 0.0f ? min(126, 14 - ilogbf(most)) : 0;
}

// h (rows of a stride of STRIDE floats, float16's scaled) as fragments of N terms.
template <typename T, int RP, int MT, int N, int STRIDE>
__device__ __forceinline__ void make_fragments(const float *h, uint4 (*frag)[MT][RP / 16][32]) {
  constexpr int KS = RP / 16;
  for (int i = threadIdx.x; i < MT * KS * 32; i += kLoraThreads) {
    const int l = i % 32, ks = i / 32 % KS, m = i / (32 * KS);
    const int c = RP == 16 ? l % 4 * 4 : ks / 2 * 32 + l % 4 * 8 + ks % 2 * 4;
    const float4 v0 = *reinterpret_cast<const float4 *>(h + (m * 16 + l / 4) * STRIDE + c);
    const float4 v1 = *reinterpret_cast<const float4 *>(h + (m * 16 + l / 4 + 8) * STRIDE + c);
    uint32_t f[N][4];
    terms_of<T, N>(v0.x, v0.y, &f[0][0], 4);
    terms_of<T, N>(v1.x, v1.y, &f[0][1], 4);
    terms_of<T, N>(v0.z, v0.w, &f[0][2], 4);
    terms_of<T, N>(v1.z, v1.w, &f[0][3], 4);
#pragma unroll
    for (int n = 0; n < N; ++n) frag[n][m][ks][l] = make_uint4(f[n][0], f[n][1], f[n][2], f[n][3]);
  }
}

// Which of 32 output columns row g of product j's B is, and where a lane's i-th 16 bytes
// of outputs begin.
__device__ __forceinline__ int b_row(bool out32, int j, int g) {
  return out32 ? j / 2 * 16 + g / 2 * 4 + j % 2 * 2 + g % 2 : g / 2 * 8 + 2 * j + g % 2;
}
__device__ __forceinline__ int lane_col(bool out32, int i, int q) { return out32 ? i * 16 + q * 4 : q * 8; }

// How many terms of T h meets B as.  Two hold 16 bits of it for bfloat16, 22 for float16: less
// than the rounding of a 16-bit output, also where the products cancel.  (One of bfloat16 left
// outputs 1.15 to 1.35 times as far off as their rounding does.  Few tokens leave the tensor pipe
// idle and pay nothing; 8192 tokens of R = 64, 4096 x 11008, take 13 us of 107 more.)  Float32
// outputs take two of float16 or three of bfloat16 (24).
template <typename T>
__host__ __device__ constexpr int terms(bool out32) {
  return out32 && std::is_same<T, __nv_bfloat16>::value ? 3 : 2;
}

// A product's fragment of A, in registers of its own.
__device__ __forceinline__ void keep4(uint32_t (&f)[4], uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("mov.b32 %0, %4;\n mov.b32 %1, %5;\n mov.b32 %2, %6;\n mov.b32 %3, %7;"
               : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
               : "r"(a), "r"(b), "r"(c), "r"(d));
}

// Part p of the parts of `per` units, and the unit in it.
struct Cursor {
  int p, i;
  __device__ __forceinline__ Cursor(int at, int per) : p(at / per), i(at % per) {}
  __device__ __forceinline__ void next(int step, int per) {
    for (i += step; i >= per; i -= per) ++p;
  }
};

__device__ __forceinline__ void read_tokens(const LoraArgs &a, const int4 &tile, int rows, int *to) {
  const int tid = threadIdx.x;
  if (tid < rows) {
    int t = tid < tile.z ? __ldg(a.plan + 4 + 4 * a.most + tile.y + tid) : -1;
    if (tid < tile.z && (t < 0 || t >= a.T)) {
      record_bad_value(a.status);
      t = -1;
    }
    to[tid] = t;
  }
}
__device__ __forceinline__ int groups_of(const LoraArgs &a) {
  const int groups = __ldg(a.plan);
  if (groups >= 0 && groups <= a.most) return groups;
  record_bad_value(a.status);
  return 0;
}

}  // namespace
}  // namespace tp
