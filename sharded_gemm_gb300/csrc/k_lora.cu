// k_lora.cu -- low-rank adapters of many requests beside a shared projection:
//   out_r[t] = y_r[t] + (scale_a sum_p x_p[t] A_p[a]^T) B_r[a]^T,   a the token's adapter.
//
// A tile is up to 16 (or 64) tokens of one adapter, taken from the step's plan; a cluster
// of C CTAs takes it in one launch.  First the C * 8 warps split the contraction and each
// multiplies its stretch of the tokens' rows with the adapter's R rows; the parts are added
// over the warps and, through distributed shared memory, the CTAs, in a fixed order.  Then
// the warps split the output's columns: a block of 32 of them is B's 32 rows against h, added
// to y.  Nothing of h goes through memory, and each CTA's sums are the same bytes.
//
// Both products are bound by bytes (a decode step reads each adapter once, a prompt its
// tokens and outputs; 2 R operations an element): warp-level m16n8k16 products are enough,
// and their fragments come straight from memory into registers, 16 bytes a lane, because a
// contraction may go through its index in any order that both operands share.  A quad's four
// lanes hold 8 neighbouring elements each, which feed two products; output columns are dealt
// to the products so that a lane ends with 8 neighbouring ones.
//
// h is float32 and meets B as a sum of two 16-bit numbers, so 2^-16 of it is lost, less than
// an output's rounding to 16 bits and 2^-16 of the adapter's part of a float32 one.  float16
// has h scaled by a power of two first, a row's largest to below 2^15.
#include "mma16.cuh"
#include "serve.cuh"

namespace tp {
namespace {

constexpr int kWarps = 8, kLoraThreads = kWarps * 32;

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// Elements k..k+7 of a row of K 16-bit elements, zeros behind its end.
__device__ __forceinline__ uint4 load8(const uint16_t *row, int64_t k, int64_t K, bool vec) {
  if (vec) return k < K ? __ldg(reinterpret_cast<const uint4 *>(row + k)) : make_uint4(0, 0, 0, 0);
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = k + 2 * i < K ? row[k + 2 * i] : 0, hi = k + 2 * i + 1 < K ? row[k + 2 * i + 1] : 0;
    v[i] = lo | hi << 16;
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ uint2 load4(const uint16_t *row, int k, int K, bool vec) {
  if (vec) return k < K ? __ldg(reinterpret_cast<const uint2 *>(row + k)) : make_uint2(0, 0);
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = k + i < K ? row[k + i] : 0;
  return make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
}

// Eight neighbouring outputs of a row as float32, and back.
struct Out8 {
  uint32_t v[8];  // float32 bits, or 16-bit pairs in the first four
};
__device__ __forceinline__ void load_out(Out8 &o, const void *base, int64_t at, int n, int dt, bool vec) {
  if (vec) {
    if (n <= 0) return;
    const int es = dt == TP_F32 ? 4 : 2;
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(base) + at * es);
    const uint4 a = p[0];
    o.v[0] = a.x, o.v[1] = a.y, o.v[2] = a.z, o.v[3] = a.w;
    if (dt == TP_F32) {
      const uint4 b = p[1];
      o.v[4] = b.x, o.v[5] = b.y, o.v[6] = b.z, o.v[7] = b.w;
    }
    return;
  }
  if (dt == TP_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = i < n ? static_cast<const uint32_t *>(base)[at + i] : 0;
  } else {
    const uint16_t *p = static_cast<const uint16_t *>(base) + at;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = (2 * i < n ? p[2 * i] : 0) | (2 * i + 1 < n ? p[2 * i + 1] : 0) << 16;
  }
}
__device__ __forceinline__ void store_out(const Out8 &o, void *base, int64_t at, int n, int dt, bool vec) {
  if (vec) {
    if (n <= 0) return;
    const int es = dt == TP_F32 ? 4 : 2;
    uint4 *p = reinterpret_cast<uint4 *>(static_cast<char *>(base) + at * es);
    p[0] = make_uint4(o.v[0], o.v[1], o.v[2], o.v[3]);
    if (dt == TP_F32) p[1] = make_uint4(o.v[4], o.v[5], o.v[6], o.v[7]);
    return;
  }
  if (dt == TP_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) static_cast<uint32_t *>(base)[at + i] = o.v[i];
  } else {
    uint16_t *p = static_cast<uint16_t *>(base) + at;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint16_t)(o.v[i / 2] >> (i % 2 * 16));
  }
}
__device__ __forceinline__ void add_out(Out8 &o, const float (&d)[8], int dt) {
  if (dt == TP_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = __float_as_uint(__uint_as_float(o.v[i]) + d[i]);
  } else if (dt == TP_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = Half2<__nv_bfloat16>::unpack(o.v[i]);
      o.v[i] = Half2<__nv_bfloat16>::pack(y.x + d[2 * i], y.y + d[2 * i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = Half2<__half>::unpack(o.v[i]);
      o.v[i] = Half2<__half>::pack(y.x + d[2 * i], y.y + d[2 * i + 1]);
    }
  }
}

// Two values as the sum of two 16-bit numbers each.  A finite value stays one (bfloat16's
// rounding may pass its largest), and behind an infinite one comes 0, not NaN.
template <typename T>
__device__ __forceinline__ void two_terms(float a, float b, uint32_t &hi, uint32_t &lo) {
  hi = Half2<T>::pack(a, b);
  float2 h = Half2<T>::unpack(hi);
  if (isinf(h.x) || isinf(h.y)) {
    if (Half2<T>::kBf16) {
      if (isinf(h.x) && !isinf(a)) hi = (hi & 0xffff0000u) | __float_as_uint(a) >> 16;
      if (isinf(h.y) && !isinf(b)) hi = (hi & 0xffffu) | (__float_as_uint(b) & 0xffff0000u);
      h = Half2<T>::unpack(hi);
    }
    lo = Half2<T>::pack(isinf(h.x) ? 0.0f : a - h.x, isinf(h.y) ? 0.0f : b - h.y);
  } else {
    lo = Half2<T>::pack(a - h.x, b - h.y);
  }
}

// Tile `tile` of the plan, counting on from group `base` (tiles `before` it): its adapter,
// first place and tokens; false behind the last.  The same in all lanes.
__device__ __forceinline__ bool find_tile(const LoraArgs &a, int groups, int rows, int64_t tile, int &base,
                                          int64_t &before, int4 &found) {
  const int lane = threadIdx.x % 32;
  const int4 *list = reinterpret_cast<const int4 *>(a.plan + 4);
  for (; base < groups; base += 32) {
    int4 g = make_int4(-1, 0, 0, 0);
    if (base + lane < groups) {
      g = __ldg(list + base + lane);
      if (g.x >= a.n || g.y < 0 || g.z < 0 || (int64_t)g.y + g.z > a.T) {  // not a plan of this call
        g = make_int4(-1, 0, 0, 0);
        record_bad_value(a.status);
      }
    }
    const int mine = g.x < 0 && a.in_place ? 0 : (g.z + rows - 1) / rows;
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

// RP: R rounded up to 16, 32, 64 or 128; MT: blocks of 16 tokens of a tile.
template <int RP, int MT>
struct LoraShared {
  static constexpr int kRows = 16 * MT, kGroups = kWarps / MT;  // warps that split a block's contraction
  static constexpr int kStride = RP + 4;
  int token[kRows];
  float unscale[kRows];  // the power of two that a row's products are multiplied by
  float part[kGroups][kRows][kStride];  // [0] in the end: this CTA's sums, read by the others
  float h[kRows][kStride];
  uint4 hi[MT][RP / 16][32], lo[MT][RP / 16][32];  // h's fragments
};

enum { kVecX = 1, kVecB = 2, kVecY = 4 };

template <typename T, int RP, int MT>
__global__ void __launch_bounds__(kLoraThreads, RP >= 128 ? 1 : 2)
    lora_kernel(const __grid_constant__ LoraArgs a, int C, int flags) {
  typedef LoraShared<RP, MT> Shared;
  constexpr int kRows = Shared::kRows, kGroups = Shared::kGroups, NT = RP / 8, KS = RP / 16;
  extern __shared__ __align__(16) uint8_t smem[];
  Shared &sh = *reinterpret_cast<Shared *>(smem);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, q = lane % 4;
  const int rank = blockIdx.x % C, m_of = warp % MT, k_of = warp / MT;
  const bool vec_x = flags & kVecX, vec_b = flags & kVecB, vec_y = flags & kVecY;
  griddep_launch_dependents();
  griddep_wait();
  const int32_t *order = a.plan + 4 + 4 * a.most;
  int groups = __ldg(a.plan);
  if (groups < 0 || groups > a.most) {
    if (tid == 0) record_bad_value(a.status);
    groups = 0;
  }
  int base = 0;
  int64_t before = 0;
  int4 tile;
  bool read = false;  // the others' sums: they may not change theirs before all have
  for (int64_t at = blockIdx.x / C; find_tile(a, groups, kRows, at, base, before, tile); at += gridDim.x / C) {
    const int id = tile.x;
    __syncthreads();  // the last tile's tokens and fragments are read
    if (tid < kRows) {
      int t = tid < tile.z ? __ldg(order + tile.y + tid) : -1;
      if (tid < tile.z && (t < 0 || t >= a.T)) {
        record_bad_value(a.status);
        t = -1;
      }
      sh.token[tid] = t;
    }
    __syncthreads();

    if (id >= 0) {
      // ---- h: this warp's block of tokens, over its stretch of the contraction
      float acc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
      const int t0 = sh.token[m_of * 16 + g], t1 = sh.token[m_of * 16 + g + 8];
      const int64_t per = (a.K + 31) / 32, units = per * a.nx;
      const int64_t slot = rank * kGroups + k_of, u1 = units * (slot + 1) / (C * kGroups);
      int64_t u = units * slot / (C * kGroups);
      int p = (int)(u / per);
      int64_t k = (u - p * per) * 32 + q * 8;
      const uint16_t *x0, *x1, *w;
      auto begin = [&]() {
        x0 = static_cast<const uint16_t *>(a.x[p]) + (int64_t)max(t0, 0) * a.ldx;
        x1 = static_cast<const uint16_t *>(a.x[p]) + (int64_t)max(t1, 0) * a.ldx;
        w = static_cast<const uint16_t *>(a.a[p]) + ((int64_t)id * a.R + g) * a.K;
      };
      if (u < u1) begin();
      const uint4 zero = make_uint4(0, 0, 0, 0);
      for (; u < u1; ++u) {
        const uint4 r0 = t0 >= 0 ? load8(x0, k, a.K, vec_x) : zero, r1 = t1 >= 0 ? load8(x1, k, a.K, vec_x) : zero;
        uint4 v[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) v[j] = j * 8 + g < a.R ? load8(w + (int64_t)j * 8 * a.K, k, a.K, vec_x) : zero;
        const uint32_t f0[4] = {r0.x, r1.x, r0.y, r1.y}, f1[4] = {r0.z, r1.z, r0.w, r1.w};
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma16816<T>(acc[j], f0, v[j].x, v[j].y);
          mma16816<T>(acc[j], f1, v[j].z, v[j].w);
        }
        k += 32;
        if (k - q * 8 >= per * 32 && u + 1 < u1) {
          ++p, k = q * 8;
          begin();
        }
      }
      if (read && C > 1) cluster_wait();
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float *to = &sh.part[k_of][m_of * 16 + g][j * 8 + q * 2];
        *reinterpret_cast<float2 *>(to) = make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2 *>(to + 8 * Shared::kStride) = make_float2(acc[j][2], acc[j][3]);
      }
      __syncthreads();
      // ---- its parts added over the warps, then over the CTAs
      constexpr int kQuads = kRows * RP / 4;
      for (int i = tid; i < kQuads; i += kLoraThreads) {
        const int row = i / (RP / 4), c = i % (RP / 4) * 4;
        float4 sum = *reinterpret_cast<const float4 *>(&sh.part[0][row][c]);
#pragma unroll
        for (int j = 1; j < kGroups; ++j) sum = add4(sum, *reinterpret_cast<const float4 *>(&sh.part[j][row][c]));
        *reinterpret_cast<float4 *>(&sh.part[0][row][c]) = sum;
      }
      if (C > 1) cluster_sync_all(); else __syncthreads();
      const float scale = a.scales ? __ldg(a.scales + id) : 1.0f;
      for (int i = tid; i < kQuads; i += kLoraThreads) {
        const int row = i / (RP / 4), c = i % (RP / 4) * 4;
        const uint32_t mine = smem_u32(&sh.part[0][row][c]);
        float4 sum = make_float4(0, 0, 0, 0);
        for (int r = 0; r < C; ++r)
          sum = add4(sum, C > 1 ? ld_cluster_f4(mapa_shared(mine, r))
                                : *reinterpret_cast<const float4 *>(&sh.part[0][row][c]));
        *reinterpret_cast<float4 *>(&sh.h[row][c]) =
            make_float4(sum.x * scale, sum.y * scale, sum.z * scale, sum.w * scale);
      }
      if (C > 1) cluster_arrive();
      read = true;
      __syncthreads();
      if (!Half2<T>::kBf16) {
        // a row's largest to 2^14..2^15; nothing is lost by a power of two but below the smallest float16
        for (int row = warp; row < kRows; row += kWarps) {
          float most = 0.0f;
          for (int c = lane; c < RP; c += 32) {
            const float v = fabsf(sh.h[row][c]);
            most = fmaxf(most, v <= 3.402823466e38f ? v : 0.0f);  // of the finite ones
          }
          most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
          const int e = most > 0.0f ? max(-100, min(100, 14 - ilogbf(most))) : 0;
          __syncwarp();
          for (int c = lane; c < RP; c += 32) sh.h[row][c] = ldexpf(sh.h[row][c], e);
          if (lane == 0) sh.unscale[row] = ldexpf(1.0f, -e);
        }
        __syncthreads();
      }
      for (int i = tid; i < MT * KS * 32; i += kLoraThreads) {
        const int l = i % 32, ks = i / 32 % KS, m = i / (32 * KS);
        const int c = RP == 16 ? l % 4 * 4 : ks / 2 * 32 + l % 4 * 8 + ks % 2 * 4;
        const float4 v0 = *reinterpret_cast<const float4 *>(&sh.h[m * 16 + l / 4][c]);
        const float4 v1 = *reinterpret_cast<const float4 *>(&sh.h[m * 16 + l / 4 + 8][c]);
        uint4 hi, lo;
        two_terms<T>(v0.x, v0.y, hi.x, lo.x);
        two_terms<T>(v1.x, v1.y, hi.y, lo.y);
        two_terms<T>(v0.z, v0.w, hi.z, lo.z);
        two_terms<T>(v1.z, v1.w, hi.w, lo.w);
        sh.hi[m][ks][l] = hi;
        sh.lo[m][ks][l] = lo;
      }
      __syncthreads();
    }

    // ---- the outputs: 32 columns a warp at a time
    const int64_t per = (a.O + 31) / 32, blocks = per * a.ny;
    for (int64_t blk = rank * kWarps + warp; blk < blocks; blk += C * kWarps) {
      const int p = (int)(blk / per);
      const int64_t c0 = (blk - p * per) * 32, cols = a.O - c0;
      uint32_t w[4][KS][2];
      if (id >= 0) {
        const uint16_t *b = static_cast<const uint16_t *>(a.b[p]) + ((int64_t)id * a.O + c0) * a.R;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int col = (g >> 1) * 8 + 2 * j + (g & 1);
          const uint16_t *row = b + (int64_t)col * a.R;
          const int R = col < cols ? a.R : 0;
          if (RP == 16) {
            const uint2 v = load4(row, q * 4, R, vec_b);
            w[j][0][0] = v.x, w[j][0][1] = v.y;
          } else {
#pragma unroll
            for (int s = 0; s < KS / 2; ++s) {
              const uint4 v = load8(row, s * 32 + q * 8, R, vec_b);
              w[j][2 * s][0] = v.x, w[j][2 * s][1] = v.y, w[j][2 * s + 1][0] = v.z, w[j][2 * s + 1][1] = v.w;
            }
          }
        }
      }
      const int64_t col = c0 + q * 8;
      const int n = (int)(a.O - col < 8 ? a.O - col : 8);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int t0 = sh.token[m * 16 + g], t1 = sh.token[m * 16 + g + 8];
        Out8 y0, y1;
        if (t0 >= 0) load_out(y0, a.y[p], t0 * a.ldy + col, n, a.out_dt, vec_y);
        if (t1 >= 0) load_out(y1, a.y[p], t1 * a.ldy + col, n, a.out_dt, vec_y);
        if (id >= 0) {
          float d[4][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.0f;
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            const uint4 h = sh.hi[m][s][lane], l = sh.lo[m][s][lane];
            const uint32_t hf[4] = {h.x, h.y, h.z, h.w}, lf[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              mma16816<T>(d[j], hf, w[j][s][0], w[j][s][1]);
              mma16816<T>(d[j], lf, w[j][s][0], w[j][s][1]);
            }
          }
          float d0[8], d1[8];
          const float f0 = Half2<T>::kBf16 ? 1.0f : sh.unscale[m * 16 + g];
          const float f1 = Half2<T>::kBf16 ? 1.0f : sh.unscale[m * 16 + g + 8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            d0[2 * j] = d[j][0] * f0, d0[2 * j + 1] = d[j][1] * f0;
            d1[2 * j] = d[j][2] * f1, d1[2 * j + 1] = d[j][3] * f1;
          }
          if (t0 >= 0) add_out(y0, d0, a.out_dt);
          if (t1 >= 0) add_out(y1, d1, a.out_dt);
        }
        if (t0 >= 0) store_out(y0, a.out[p], t0 * a.ldo + col, n, a.out_dt, vec_y);
        if (t1 >= 0) store_out(y1, a.out[p], t1 * a.ldo + col, n, a.out_dt, vec_y);
      }
    }
  }
  if (read && C > 1) cluster_wait();  // no CTA leaves while another may still read its shared memory
}

// The same on the CUDA cores, a block a token: the cross-check.
__device__ __forceinline__ float in16(const void *p, int64_t i, int dt) {
  return dt == TP_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i])
                       : __half2float(static_cast<const __half *>(p)[i]);
}
__global__ void __launch_bounds__(256) lora_simt_kernel(const __grid_constant__ LoraArgs a) {
  __shared__ float h[128];
  __shared__ int adapter, token;
  griddep_wait();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) adapter = token = -1;
  __syncthreads();
  const int groups = min((int64_t)max(a.plan[0], 0), a.most);
  for (int i = tid; i < groups; i += 256) {
    const int32_t *g = a.plan + 4 + 4 * i;
    if (blockIdx.x >= (unsigned)g[1] && (int64_t)blockIdx.x < (int64_t)g[1] + g[2])
      adapter = g[0], token = a.plan[4 + 4 * a.most + blockIdx.x];
  }
  __syncthreads();
  const int id = adapter, t = token;
  if (t < 0 || (id < 0 && a.in_place)) return;
  if (t >= a.T || id >= a.n) {
    if (tid == 0) record_bad_value(a.status);
    return;
  }
  if (id >= 0)
    for (int r = warp; r < a.R; r += 8) {
      float sum = 0.0f;
      for (int p = 0; p < a.nx; ++p)
        for (int64_t k = lane; k < a.K; k += 32)
          sum += in16(a.x[p], t * a.ldx + k, a.dt) * in16(a.a[p], ((int64_t)id * a.R + r) * a.K + k, a.dt);
#pragma unroll
      for (int m = 16; m > 0; m /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
      if (lane == 0) h[r] = sum * (a.scales ? a.scales[id] : 1.0f);
    }
  __syncthreads();
  for (int p = 0; p < a.ny; ++p)
    for (int64_t c = tid; c < a.O; c += 256) {
      float sum = 0.0f;
      if (id >= 0)
        for (int r = 0; r < a.R; ++r) sum += h[r] * in16(a.b[p], ((int64_t)id * a.O + c) * a.R + r, a.dt);
      const int64_t i = t * a.ldy + c, o = t * a.ldo + c;
      if (a.out_dt == TP_F32) {
        static_cast<float *>(a.out[p])[o] = static_cast<const float *>(a.y[p])[i] + sum;
      } else if (a.out_dt == TP_BF16) {
        static_cast<__nv_bfloat16 *>(a.out[p])[o] =
            id < 0 ? static_cast<const __nv_bfloat16 *>(a.y[p])[i] : __float2bfloat16(in16(a.y[p], i, TP_BF16) + sum);
      } else {
        static_cast<__half *>(a.out[p])[o] =
            id < 0 ? static_cast<const __half *>(a.y[p])[i] : __float2half(in16(a.y[p], i, TP_F16) + sum);
      }
    }
}

bool all_aligned(const void *const *p, int n, int to) {
  for (int i = 0; i < n; ++i)
    if ((uintptr_t)p[i] % to) return false;
  return true;
}

template <typename T, int RP, int MT>
int launch(const LoraArgs &a, int C, int64_t tiles, int flags, cudaStream_t s) {
  auto kern = lora_kernel<T, RP, MT>;
  const size_t smem = sizeof(LoraShared<RP, MT>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return cuda_error(e, "adapter launch");
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)(tiles * C));
  cfg.blockDim = dim3(kLoraThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, a, C, flags);
  if (e != cudaSuccess) return cuda_error(e, "adapter launch");
  note_launch();
  return TP_OK;
}

template <typename T>
int launch(const LoraArgs &a, cudaStream_t s) {
  const int es = a.out_dt == TP_F32 ? 4 : 2, RP = a.R <= 16 ? 16 : a.R <= 32 ? 32 : a.R <= 64 ? 64 : 128;
  int flags = 0;
  if (a.K % 8 == 0 && (a.ldx % 8 == 0 || a.T == 1) && all_aligned(a.x, a.nx, 16) && all_aligned(a.a, a.nx, 16))
    flags |= kVecX;
  if (a.R % (RP == 16 ? 4 : 8) == 0 && all_aligned(a.b, a.ny, RP == 16 ? 8 : 16)) flags |= kVecB;
  if (a.O % 8 == 0 && ((a.ldy * es % 16 == 0 && a.ldo * es % 16 == 0) || a.T == 1) && all_aligned(a.y, a.ny, 16) &&
      all_aligned(a.out, a.ny, 16))
    flags |= kVecY;
  const bool small = a.T <= 1024;
  const int rows = small ? 16 : 64, C = 8;
  int64_t tiles = a.T / rows + a.most;
  if (tiles > (1 << 20)) tiles = 1 << 20;
#define TP_LORA(RP) \
  case RP: return small ? launch<T, RP, 1>(a, C, tiles, flags, s) : launch<T, RP, 4>(a, C, tiles, flags, s);
  switch (RP) {
    TP_LORA(16)
    TP_LORA(32)
    TP_LORA(64)
    default:
    TP_LORA(128)
  }
#undef TP_LORA
}

}  // namespace

int launch_lora(const LoraArgs &a, cudaStream_t s) {
  return a.dt == TP_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

int launch_lora_simt(const LoraArgs &a, cudaStream_t s) {
  const cudaError_t e = launch_pdl(lora_simt_kernel, dim3((unsigned)a.T), dim3(256), 0, s, a);
  if (e != cudaSuccess) return cuda_error(e, "adapter launch");
  note_launch();
  return TP_OK;
}

}  // namespace tp
