// k_lora.cu -- low-rank adapters of many requests beside a shared projection:
//   out_r[t] = y_r[t] + (scale_a sum_p x_p[t] A_p[a]^T) B_r[a]^T,   a the token's adapter.
//
// This file: steps of few tokens, operands without 16-byte alignment, and the CUDA-core
// cross-check; prompts are k_loraprompt.cu's.  A tile is up to 16 tokens of one adapter,
// taken from the step's plan; C CTAs of a cluster of 8 take it in one launch.  First their
// C * 8 warps split the contraction and each multiplies its stretch of the tokens' rows with
// the adapter's R rows; the parts are added over the warps and, through distributed shared
// memory, the CTAs, in a fixed order.  Then the warps split the output's columns: 32 of them
// are B's 32 rows against h, added to y.  Nothing of h goes through memory.  The more tiles
// the plan holds, the fewer CTAs take one (8, 4, 2, 1), so that all run at once.
//
// Bound by bytes (each adapter is read once) and, of one token, by latency: 2 R operations
// an element are few, so warp-level products do.
//
// Measured: one token, R = 16, 4096 x 12288 on 8 ranks 5.6 us; 64 tokens of 47 adapters 12.5
// (28 MB, 4.2 at the copy rate); 97 tokens of 33 adapters, R = 32, 4096 x 4096, float32 11.0.
#include <atomic>

#include "lora.cuh"

namespace tp {
namespace {

// Elements k..k+7 of a row of K 16-bit elements, zeros behind its end.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t *row, int k, int K) {
  if (VEC) return k < K ? __ldg(reinterpret_cast<const uint4 *>(row + k)) : make_uint4(0, 0, 0, 0);
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = k + 2 * i < K ? row[k + 2 * i] : 0, hi = k + 2 * i + 1 < K ? row[k + 2 * i + 1] : 0;
    v[i] = lo | hi << 16;
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
template <bool VEC>
__device__ __forceinline__ uint2 load4(const uint16_t *row, int k, int K) {
  if (VEC) return k < K ? __ldg(reinterpret_cast<const uint2 *>(row + k)) : make_uint2(0, 0);
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = k + i < K ? row[k + i] : 0;
  return make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
}

// A lane's eight outputs of a row, at `col` and, float32, the second four 16 columns on:
// float32 bits, or 16-bit pairs.  Columns of `cols` and more are not there.
template <bool OUT32>
struct Out8 {
  uint32_t v[OUT32 ? 8 : 4];
};
template <bool VEC, bool OUT32>
__device__ __forceinline__ void load_out(Out8<OUT32> &o, const void *base, int64_t row, int col, int cols) {
  constexpr int kEach = OUT32 ? 4 : 8;  // columns of 16 bytes
#pragma unroll
  for (int i = 0; i < 8 / kEach; ++i) {
    const int at = col + i * 16;
    if (VEC) {
      if (at >= cols) continue;
      const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const char *>(base) + (row + at) * (16 / kEach));
      o.v[4 * i] = a.x, o.v[4 * i + 1] = a.y, o.v[4 * i + 2] = a.z, o.v[4 * i + 3] = a.w;
    } else if constexpr (OUT32) {
#pragma unroll
      for (int k = 0; k < 4; ++k) o.v[4 * i + k] = at + k < cols ? static_cast<const uint32_t *>(base)[row + at + k] : 0;
    } else {
      const uint16_t *p = static_cast<const uint16_t *>(base) + row + at;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        o.v[k] = (at + 2 * k < cols ? p[2 * k] : 0) | (at + 2 * k + 1 < cols ? p[2 * k + 1] : 0) << 16;
    }
  }
}
template <bool VEC, bool OUT32>
__device__ __forceinline__ void store_out(const Out8<OUT32> &o, void *base, int64_t row, int col, int cols) {
  constexpr int kEach = OUT32 ? 4 : 8;
#pragma unroll
  for (int i = 0; i < 8 / kEach; ++i) {
    const int at = col + i * 16;
    if (VEC) {
      if (at < cols)
        *reinterpret_cast<uint4 *>(static_cast<char *>(base) + (row + at) * (16 / kEach)) =
            make_uint4(o.v[4 * i], o.v[4 * i + 1], o.v[4 * i + 2], o.v[4 * i + 3]);
    } else if constexpr (OUT32) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (at + k < cols) static_cast<uint32_t *>(base)[row + at + k] = o.v[4 * i + k];
    } else {
      uint16_t *p = static_cast<uint16_t *>(base) + row + at;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (at + k < cols) p[k] = (uint16_t)(o.v[k / 2] >> (k % 2 * 16));
    }
  }
}
template <bool OUT32>
__device__ __forceinline__ void add_out(Out8<OUT32> &o, const float (&d)[8], bool bf16) {
  if constexpr (OUT32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = __float_as_uint(__uint_as_float(o.v[i]) + d[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = bf16 ? Half2<__nv_bfloat16>::unpack(o.v[i]) : Half2<__half>::unpack(o.v[i]);
      const float a = y.x + d[2 * i], b = y.y + d[2 * i + 1];
      o.v[i] = bf16 ? Half2<__nv_bfloat16>::pack(a, b) : Half2<__half>::pack(a, b);
    }
  }
}

// RP: R rounded up to 16, 32, 64 or 128.
template <typename T, int RP>
struct LoraShared {
  static constexpr int kStride = RP + 4;
  uint4 frag[terms<T>(true)][1][RP / 16][32];
  float part[kWarps][16][kStride];  // [0] in the end: this CTA's sums, read by the others
  float h[16][kStride];
  int token[16];
  float unscale[16];  // the power of two that a row's products are multiplied by
};

constexpr int kCluster = 8;
template <int RP>
constexpr int kResident = RP == 128 ? 1 : RP == 16 ? 3 : 2;  // CTAs an SM

// The tiles of a call, C of a cluster's CTAs each.  With all eight, S clusters may share a
// tile, each with h for itself and a share of the columns.  CTAs of one cluster go through
// the same turns, those without a tile in the last one too.
template <typename T, int RP, bool VEC, bool OUT32, int C>
__device__ __forceinline__ void lora_tiles(const LoraArgs &a, int groups, int S) {
  typedef LoraShared<T, RP> Shared;
  constexpr int NT = RP / 8, KS = RP / 16, kStride = Shared::kStride, kTerms = terms<T>(OUT32);
  extern __shared__ __align__(16) uint8_t smem[];
  Shared &sh = *reinterpret_cast<Shared *>(smem);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, q = lane % 4;
  const int K = (int)a.K, O = (int)a.O;
  const int per_k = (K + 31) / 32, units = per_k * a.nx;
  const int per_o = (O + 31) / 32, blocks = per_o * a.ny;
  const bool out_bf16 = a.out_dt == TP_BF16;
  constexpr int kSubs = kCluster / C;
  const int in = blockIdx.x % kCluster, rank = in % C, sub = in / C, cluster = blockIdx.x / kCluster;
  const int step = S * C * kWarps, blk0 = (cluster % S * C + rank) * kWarps + warp, u0 = rank * kWarps + warp;
  int base = 0;
  int64_t before = 0;
  int4 tile;
  bool read = false;  // the others' sums: they may not change theirs before all have
  for (int64_t first = cluster / S * kSubs;; first += gridDim.x / kCluster / S * kSubs) {
    if (!find_tile(a, groups, 16, !a.in_place, first + sub, base, before, tile)) {
      if (kSubs == 1 || C == 1 || first >= before) break;
      tile = make_int4(-1, 0, 0, 0);
    }
    const int id = tile.x;
    __syncthreads();  // the last tile's tokens and fragments are read
    read_tokens(a, tile, 16, sh.token);
    __syncthreads();
    const int t0 = sh.token[g], t1 = sh.token[g + 8];

    // ---- a block's rows of B, and the old outputs
    struct Block {
      uint32_t w[4][KS][2];
      Out8<OUT32> y0, y1;
    };
    auto fetch = [&](const Cursor &c, Block &o) {
      const int col = c.i * 32 + lane_col(OUT32, 0, q);
      if (id >= 0) {
        const uint16_t *b = static_cast<const uint16_t *>(a.b[c.p]) + ((int64_t)id * O + c.i * 32) * a.R;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = b_row(OUT32, j, g);
          const uint16_t *row = b + r * a.R;
          const int R = c.i * 32 + r < O ? a.R : 0;
          if (RP == 16) {
            const uint2 v = load4<VEC>(row, q * 4, R);
            o.w[j][0][0] = v.x, o.w[j][0][1] = v.y;
          } else {
#pragma unroll
            for (int s = 0; s < KS / 2; ++s) {
              const uint4 v = load8<VEC>(row, s * 32 + q * 8, R);
              o.w[j][2 * s][0] = v.x, o.w[j][2 * s][1] = v.y, o.w[j][2 * s + 1][0] = v.z, o.w[j][2 * s + 1][1] = v.w;
            }
          }
        }
      }
      if (t0 >= 0) load_out<VEC>(o.y0, a.y[c.p], t0 * a.ldy, col, O);
      if (t1 >= 0) load_out<VEC>(o.y1, a.y[c.p], t1 * a.ldy, col, O);
    };
    // (One block ahead, in registers: with two or three there, as many CTAs an SM do not fit, which
    // costs more: 13.7 us for 64 tokens of 50 adapters against 15.4 and 21.  Rings in shared memory,
    // as k_loraprompt.cu has, would take no registers and have not been tried here.)
    Block now;
    Cursor c(blk0, per_o);

    if (id >= 0) {
      // ---- h: this warp's stretch of the contraction
      float acc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      Cursor cu(u0, per_k);
#pragma unroll (RP < 64 ? 2 : 1)  // (R = 64: two spill, 22.5 us where one takes 19.5)
      for (int u = u0; u < units; u += C * kWarps) {  // neighbours read a row's neighbouring bytes
        const int k = cu.i * 32 + q * 8;
        const uint16_t *x = static_cast<const uint16_t *>(a.x[cu.p]);
        const uint16_t *w = static_cast<const uint16_t *>(a.a[cu.p]) + ((int64_t)id * a.R + g) * K;
        const uint4 r0 = t0 >= 0 ? load8<VEC>(x + t0 * a.ldx, k, K) : zero;
        const uint4 r1 = t1 >= 0 ? load8<VEC>(x + t1 * a.ldx, k, K) : zero;
        uint4 v[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) v[j] = j * 8 + g < a.R ? load8<VEC>(w + (int64_t)j * 8 * K, k, K) : zero;
        uint32_t f0[4], f1[4];
        keep4(f0, r0.x, r1.x, r0.y, r1.y);
        keep4(f1, r0.z, r1.z, r0.w, r1.w);
#pragma unroll
        for (int j = 0; j < NT; ++j) mma16816<T>(acc[j], f0, v[j].x, v[j].y);
#pragma unroll
        for (int j = 0; j < NT; ++j) mma16816<T>(acc[j], f1, v[j].z, v[j].w);
        cu.next(C * kWarps, per_k);
      }
      if (blk0 < blocks) fetch(c, now);  // under the sums' exchange
      if (read) cluster_wait();
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float *to = &sh.part[warp][g][j * 8 + q * 2];
        *reinterpret_cast<float2 *>(to) = make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2 *>(to + 8 * kStride) = make_float2(acc[j][2], acc[j][3]);
      }
      __syncthreads();
      // ---- its parts added over the warps, then over the CTAs
      for (int i = tid; i < 4 * RP; i += kLoraThreads) {
        const int row = i / (RP / 4), col = i % (RP / 4) * 4;
        float4 sum = *reinterpret_cast<const float4 *>(&sh.part[0][row][col]);
#pragma unroll
        for (int j = 1; j < kWarps; ++j) sum = add4(sum, *reinterpret_cast<const float4 *>(&sh.part[j][row][col]));
        *reinterpret_cast<float4 *>(&sh.part[0][row][col]) = sum;
      }
      if (C > 1)
        cluster_sync_all();
      else
        __syncthreads();
      const float scale = a.scales ? __ldg(a.scales + id) : 1.0f;
      for (int i = tid; i < 4 * RP; i += kLoraThreads) {
        const int row = i / (RP / 4), col = i % (RP / 4) * 4;
        const uint32_t mine = smem_u32(&sh.part[0][row][col]);
        float4 of[C], sum = make_float4(0, 0, 0, 0);  // all asked for before the first is added
#pragma unroll
        for (int r = 0; r < C; ++r) of[r] = ld_cluster_f4(mapa_shared(mine, sub * C + r));
#pragma unroll
        for (int r = 0; r < C; ++r) sum = add4(sum, of[r]);
        *reinterpret_cast<float4 *>(&sh.h[row][col]) = scaled_h(sum, scale, col, a.R);
      }
      if (C > 1) cluster_arrive();
      read = C > 1;
      __syncthreads();
      if (!Half2<T>::kBf16) {
        for (int row = warp; row < 16; row += kWarps) {
          const int e = row_exponent<RP>(sh.h[row]);
          __syncwarp();
          for (int col = lane; col < RP; col += 32) sh.h[row][col] = ldexpf(sh.h[row][col], e);
          if (lane == 0) sh.unscale[row] = ldexpf(1.0f, -e);
        }
        __syncthreads();
      }
      make_fragments<T, RP, 1, kTerms, kStride>(&sh.h[0][0], sh.frag);
      __syncthreads();
    } else {
      if (tile.z > 0 && blk0 < blocks) fetch(c, now);
      if (kSubs > 1 && C > 1) {
        if (read) cluster_wait();
        cluster_sync_all();
        cluster_arrive();
        read = true;
      }
    }

    // ---- the outputs: 32 columns a warp at a time
    const float f0 = Half2<T>::kBf16 || id < 0 ? 1.0f : sh.unscale[g];
    const float f1 = Half2<T>::kBf16 || id < 0 ? 1.0f : sh.unscale[g + 8];
    for (int blk = tile.z > 0 ? blk0 : blocks; blk < blocks; blk += step) {
      const int p = c.p, col = c.i * 32 + lane_col(OUT32, 0, q);
      c.next(step, per_o);
      if (id >= 0) {
        float d[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int i = 0; i < kTerms; ++i) {
            const uint4 f = sh.frag[i][0][s][lane];
            const uint32_t hf[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) mma16816<T>(d[j], hf, now.w[j][s][0], now.w[j][s][1]);
          }
        float add0[8], add1[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          add0[2 * j] = d[j][0] * f0, add0[2 * j + 1] = d[j][1] * f0;
          add1[2 * j] = d[j][2] * f1, add1[2 * j + 1] = d[j][3] * f1;
        }
        add_out(now.y0, add0, out_bf16);
        add_out(now.y1, add1, out_bf16);
      }
      const Out8<OUT32> y0 = now.y0, y1 = now.y1;
      if (blk + step < blocks) fetch(c, now);
      if (t0 >= 0) store_out<VEC>(y0, a.out[p], t0 * a.ldo, col, O);
      if (t1 >= 0) store_out<VEC>(y1, a.out[p], t1 * a.ldo, col, O);
    }
  }
  if (read) cluster_wait();  // no CTA leaves while another may still read its shared memory
}

template <typename T, int RP, bool VEC, bool OUT32>
__global__ void __launch_bounds__(kLoraThreads, kResident<RP>)
    lora_kernel(const __grid_constant__ LoraArgs a, int S) {
  griddep_launch_dependents();
  griddep_wait();
  lora_tiles<T, RP, VEC, OUT32, kCluster>(a, groups_of(a), S);
}

// More tiles than clusters run at once, if the plan has as many as it may: it says how many
// CTAs take one.  (4096 x 4096, microseconds with 8 CTAs a tile | with as many as fit:
// R = 16, 256 tokens of 152 adapters 38 | 22, 1024 of 249 66 | 38; R = 64, 64 tokens of 40
// adapters 30 | 19, 1024 of 249 143 | 60; R = 128 and 93 adapters 99 | 60.)
template <typename T, int RP, bool OUT32>
__global__ void __launch_bounds__(kLoraThreads, kResident<RP>) lora_many_kernel(const __grid_constant__ LoraArgs a, int) {
  griddep_launch_dependents();
  griddep_wait();
  // About so many tiles: the groups of an adapter's few tokens are one each.
  const int groups = groups_of(a), clusters = gridDim.x / kCluster, all = (int)a.T;
  const int with = max(0, min(all, __ldg(a.plan + 1))), adapters = groups - (with < all);
  const int tiles = adapters + max(0, with - 8 * adapters) / 16 + (a.in_place ? 0 : (all - with + 15) / 16);
  if (tiles <= clusters)
    lora_tiles<T, RP, true, OUT32, 8>(a, groups, 1);
  else if (tiles <= 2 * clusters)
    lora_tiles<T, RP, true, OUT32, 4>(a, groups, 1);
  else if (RP == 128 || tiles <= 4 * clusters)
    lora_tiles<T, RP, true, OUT32, 2>(a, groups, 1);
  else
    lora_tiles<T, RP, true, OUT32, 1>(a, groups, 1);
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

template <typename T, int RP, bool VEC, bool OUT32>
int launch(const LoraArgs &a, cudaStream_t s) {
  void (*kern)(LoraArgs, int) = lora_kernel<T, RP, VEC, OUT32>;
  const size_t smem = sizeof(LoraShared<T, RP>);
  cudaError_t e = cudaSuccess;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.blockDim = dim3(kLoraThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  static std::atomic<int> resident[64];  // clusters
  int device = 0;
  cudaGetDevice(&device);
  int wave = resident[device &= 63].load(std::memory_order_relaxed);
  if (!wave) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if constexpr (VEC)
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(lora_many_kernel<T, RP, OUT32>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    cfg.gridDim = dim3(kCluster);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&wave, kern, &cfg);
    if (e != cudaSuccess) return cuda_error(e, "adapter launch");
    if (wave < 1) wave = 1;
    resident[device].store(wave, std::memory_order_relaxed);
  }
  const int64_t tiles = a.T / 16 + a.most, blocks = (a.O + 31) / 32 * a.ny;  // at most
  const int64_t most = (blocks + kCluster * kWarps - 1) / (kCluster * kWarps), room = wave / tiles;
  const int S = (int)(room < 1 ? 1 : room < most ? room : most);
  if constexpr (VEC)
    if (tiles > wave) kern = lora_many_kernel<T, RP, OUT32>;
  // (Operands without alignment, which come here in steps of any size: a cluster a tile, 135 us
  // for 5000 tokens of R = 32, 1663 x 1511, where one wave's clusters in turns take 191.)
  const int64_t at_once = VEC ? wave : 1 << 20;
  cfg.gridDim = dim3((unsigned)((tiles * S < at_once ? tiles * S : at_once) * kCluster));
  e = cudaLaunchKernelEx(&cfg, kern, a, S);
  if (e != cudaSuccess) return cuda_error(e, "adapter launch");
  note_launch();
  return TP_OK;
}

template <typename T, int RP, bool VEC>
int launch(const LoraArgs &a, cudaStream_t s) {
  return a.out_dt == TP_F32 ? launch<T, RP, VEC, true>(a, s) : launch<T, RP, VEC, false>(a, s);
}

template <typename T, bool VEC>
int launch(const LoraArgs &a, int RP, cudaStream_t s) {
  switch (RP) {
    case 16: return launch<T, 16, VEC>(a, s);
    case 32: return launch<T, 32, VEC>(a, s);
    case 64: return launch<T, 64, VEC>(a, s);
    default: return launch<T, 128, VEC>(a, s);
  }
}

}  // namespace

int launch_lora(const LoraArgs &a, cudaStream_t s) {
  const int es = a.out_dt == TP_F32 ? 4 : 2, RP = a.R <= 16 ? 16 : a.R <= 32 ? 32 : a.R <= 64 ? 64 : 128;
  const bool vec = a.K % 8 == 0 && (a.ldx % 8 == 0 || a.T == 1) && all_aligned(a.x, a.nx, 16) && all_aligned(a.a, a.nx, 16) &&
                   a.R % (RP == 16 ? 4 : 8) == 0 && all_aligned(a.b, a.ny, RP == 16 ? 8 : 16) && a.O % 8 == 0 &&
                   ((a.ldy * es % 16 == 0 && a.ldo * es % 16 == 0) || a.T == 1) && all_aligned(a.y, a.ny, 16) &&
                   all_aligned(a.out, a.ny, 16);
  if (vec && a.workspace) return launch_lora_prompt(a, RP, s);
  if (a.dt == TP_BF16)
    return vec ? launch<__nv_bfloat16, true>(a, RP, s) : launch<__nv_bfloat16, false>(a, RP, s);
  return vec ? launch<__half, true>(a, RP, s) : launch<__half, false>(a, RP, s);
}

int launch_lora_simt(const LoraArgs &a, cudaStream_t s) {
  const cudaError_t e = launch_pdl(lora_simt_kernel, dim3((unsigned)a.T), dim3(256), 0, s, a);
  if (e != cudaSuccess) return cuda_error(e, "adapter launch");
  note_launch();
  return TP_OK;
}

}  // namespace tp
