// k_loraprompt.cu -- the adapters of k_lora.cu for steps of many tokens, as two passes:
//   h[i] = scale_a sum_p x_p[t] A_p[a]^T   for the token t at place i of the plan,
//   out_r[t] = y_r[t] + h[i] B_r[a]^T,
// h float32 in the call's workspace.  A tile is up to 64 tokens of one adapter.
//
// Bound by bytes: the tokens' rows once, the outputs' once in and once out, an adapter once a
// tile from L2.  So both passes are streams whose loads run ahead: each lane copies what it
// alone will read into its part of a ring in shared memory (16-byte asynchronous copies), with
// no barrier between the copy and its use.  (As one kernel, h exchanged within a cluster, the
// barriers between the products stood in the way of the streams, and registers for both were
// too many: 309 us for 8192 tokens, R = 64, 4096 x 11008, where 66 us of bytes move.)
#include "lora.cuh"

namespace tp {
namespace {

constexpr int kTile = 64;

// ---------------------------------------------------------------- the first pass
// Eight warps: kM groups of MW blocks of 16 tokens, kG stretches of the contraction.
template <int RP>
struct ShrinkShared {
  static constexpr int MW = RP == 128 ? 1 : 2, kM = 4 / MW, kG = kWarps / kM, kStride = RP + 4;
  static constexpr int kAhead = 4;  // units
  union {
    uint4 ring[kWarps][kAhead][MW * 2][32];
    float part[kG][kTile][kStride];  // [0] in the end: this CTA's sums, read by the others
  };
  int token[kTile];
};

template <typename T, int RP>
__global__ void __launch_bounds__(kLoraThreads, RP == 128 ? 1 : 2)
    lora_shrink_kernel(const __grid_constant__ LoraArgs a, int C) {
  typedef ShrinkShared<RP> Shared;
  constexpr int NT = RP / 8, MW = Shared::MW, kG = Shared::kG, kAhead = Shared::kAhead, kStride = Shared::kStride;
  extern __shared__ __align__(16) uint8_t smem[];
  Shared &sh = *reinterpret_cast<Shared *>(smem);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, q = lane % 4;
  const int rank = blockIdx.x % C, K = (int)a.K, per = (K + 31) / 32, units = per * a.nx;
  const int m0 = warp % Shared::kM * MW, slot = rank * kG + warp / Shared::kM;
  const int u0 = (int)((int64_t)units * slot / (C * kG)), u1 = (int)((int64_t)units * (slot + 1) / (C * kG));
  uint4 *const ring = &sh.ring[warp][0][0][lane];
  griddep_launch_dependents();
  griddep_wait();
  const int groups = groups_of(a);
  int base = 0;
  int64_t before = 0;
  int4 tile;
  for (int64_t at = blockIdx.x / C; find_tile(a, groups, kTile, at, base, before, tile); at += gridDim.x / C) {
    const int id = tile.x;
    if (id < 0) continue;  // they need no h
    if (C > 1) cluster_sync_all(); else __syncthreads();  // the last tile's sums are read
    read_tokens(a, tile, kTile, sh.token);
    __syncthreads();
    int t[MW][2];
#pragma unroll
    for (int m = 0; m < MW; ++m) t[m][0] = sh.token[(m0 + m) * 16 + g], t[m][1] = sh.token[(m0 + m) * 16 + g + 8];
    Cursor cx(u0, per), ca(u0, per);
    int ux = u0, x_slot = 0, slot_at = 0;
    auto fetch = [&]() {
      if (ux < u1) {
        const int k = cx.i * 32 + q * 8;
        const uint16_t *x = static_cast<const uint16_t *>(a.x[cx.p]);
#pragma unroll
        for (int i = 0; i < 2 * MW; ++i) {
          const int row = t[i / 2][i % 2];
          const bool valid = row >= 0 && k < K;
          cp_async16(smem_u32(ring + (x_slot * 2 * MW + i) * 32), valid ? x + row * a.ldx + k : x, valid);
        }
        cx.next(1, per);
      }
      ++ux;
      x_slot = x_slot + 1 == kAhead ? 0 : x_slot + 1;
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i) fetch();
    float acc[MW][NT][4];
#pragma unroll
    for (int m = 0; m < MW; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[m][j][0] = acc[m][j][1] = acc[m][j][2] = acc[m][j][3] = 0.0f;
    for (int u = u0; u < u1; ++u) {
      const int k = ca.i * 32 + q * 8;
      const uint16_t *w = static_cast<const uint16_t *>(a.a[ca.p]) + ((int64_t)id * a.R + g) * K + k;
      uint4 v[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j)
        v[j] = j * 8 + g < a.R && k < K ? __ldg(reinterpret_cast<const uint4 *>(w + (int64_t)j * 8 * K)) : make_uint4(0, 0, 0, 0);
      ca.next(1, per);
      cp_async_wait<kAhead - 2>();
      uint4 r[MW][2];
#pragma unroll
      for (int i = 0; i < 2 * MW; ++i) r[i / 2][i % 2] = ring[(slot_at * 2 * MW + i) * 32];
      slot_at = slot_at + 1 == kAhead ? 0 : slot_at + 1;
      fetch();
#pragma unroll
      for (int m = 0; m < MW; ++m) {
        const uint32_t f0[4] = {r[m][0].x, r[m][1].x, r[m][0].y, r[m][1].y};
        const uint32_t f1[4] = {r[m][0].z, r[m][1].z, r[m][0].w, r[m][1].w};
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma16816<T>(acc[m][j], f0, v[j].x, v[j].y);
          mma16816<T>(acc[m][j], f1, v[j].z, v[j].w);
        }
      }
    }
    cp_async_wait<0>();
    __syncthreads();  // the rings are read
#pragma unroll
    for (int m = 0; m < MW; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float *to = &sh.part[warp / Shared::kM][(m0 + m) * 16 + g][j * 8 + q * 2];
        *reinterpret_cast<float2 *>(to) = make_float2(acc[m][j][0], acc[m][j][1]);
        *reinterpret_cast<float2 *>(to + 8 * kStride) = make_float2(acc[m][j][2], acc[m][j][3]);
      }
    __syncthreads();
    // ---- the parts added over the warps, then over the CTAs, a share of the rows each
    constexpr int kQuads = kTile * RP / 4;
    if (C > 1) {
      for (int i = tid; i < kQuads; i += kLoraThreads) {
        const int row = i / (RP / 4), c = i % (RP / 4) * 4;
        float4 sum = *reinterpret_cast<const float4 *>(&sh.part[0][row][c]);
#pragma unroll
        for (int j = 1; j < kG; ++j) sum = add4(sum, *reinterpret_cast<const float4 *>(&sh.part[j][row][c]));
        *reinterpret_cast<float4 *>(&sh.part[0][row][c]) = sum;
      }
      cluster_sync_all();
    }
    const float scale = a.scales ? __ldg(a.scales + id) : 1.0f;
    for (int i = kQuads / C * rank + tid; i < kQuads / C * (rank + 1); i += kLoraThreads) {
      const int row = i / (RP / 4), c = i % (RP / 4) * 4;
      float4 sum = make_float4(0, 0, 0, 0);
      if (C > 1) {
        const uint32_t mine = smem_u32(&sh.part[0][row][c]);
        for (int r = 0; r < C; ++r) sum = add4(sum, ld_cluster_f4(mapa_shared(mine, r)));
      } else {
#pragma unroll
        for (int j = 0; j < kG; ++j) sum = add4(sum, *reinterpret_cast<const float4 *>(&sh.part[j][row][c]));
      }
      if (row < tile.z)
        *reinterpret_cast<float4 *>(a.workspace + (int64_t)(tile.y + row) * RP + c) =
            make_float4(sum.x * scale, sum.y * scale, sum.z * scale, sum.w * scale);
    }
  }
  if (C > 1) cluster_sync_all();  // no CTA leaves while another may still read its shared memory
}

// ---------------------------------------------------------------- the second pass
template <typename T, int RP, bool OUT32>
struct ExpandShared {
  static constexpr int kTerms = Half2<T>::kBf16 && OUT32 ? 3 : 2, kStride = RP + 4;
  static constexpr int kWords = OUT32 ? 2 : 1, kAhead = 6 / kWords;  // of a block of 16 tokens and 32 columns
  union {
    uint4 ring[kWarps][kAhead][2 * kWords][32];
    float h[kTile][kStride];
  };
  uint4 frag[kTerms][4][RP / 16][32];
  int token[kTile];
  float unscale[kTile];
};

template <typename T>
__device__ __forceinline__ uint4 add_pairs(uint4 y, const float *d) {
  uint32_t v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Half2<T>::unpack(v[i]);
    v[i] = Half2<T>::pack(f.x + d[2 * i], f.y + d[2 * i + 1]);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ uint4 add_floats(uint4 y, const float *d) {
  return make_uint4(__float_as_uint(__uint_as_float(y.x) + d[0]), __float_as_uint(__uint_as_float(y.y) + d[1]),
                    __float_as_uint(__uint_as_float(y.z) + d[2]), __float_as_uint(__uint_as_float(y.w) + d[3]));
}

template <typename T, int RP, bool OUT32>
__global__ void __launch_bounds__(kLoraThreads, RP == 128 ? 1 : 2)
    lora_expand_kernel(const __grid_constant__ LoraArgs a, int S) {
  typedef ExpandShared<T, RP, OUT32> Shared;
  constexpr int KS = RP / 16, kAhead = Shared::kAhead, kTerms = Shared::kTerms, kStride = Shared::kStride;
  constexpr int kWords = Shared::kWords, kSize = OUT32 ? 4 : 2;
  extern __shared__ __align__(16) uint8_t smem[];
  Shared &sh = *reinterpret_cast<Shared *>(smem);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, q = lane % 4;
  const int O = (int)a.O, per = (O + 31) / 32, blocks = per * a.ny, step = S * kWarps;
  const int blk0 = blockIdx.x % S * kWarps + warp;
  const bool out_bf16 = a.out_dt == TP_BF16;
  uint4 *const ring = &sh.ring[warp][0][0][lane];
  griddep_launch_dependents();
  griddep_wait();
  const int groups = groups_of(a);
  int base = 0;
  int64_t before = 0;
  int4 tile;
  for (int64_t at = blockIdx.x / S; find_tile(a, groups, kTile, at, base, before, tile); at += gridDim.x / S) {
    const int id = tile.x;
    __syncthreads();
    read_tokens(a, tile, kTile, sh.token);
    if (id >= 0) {
      for (int i = tid; i < kTile * RP / 4; i += kLoraThreads) {
        const int row = i / (RP / 4), c = i % (RP / 4) * 4;
        float4 v = make_float4(0, 0, 0, 0);
        if (row < tile.z) v = __ldcg(reinterpret_cast<const float4 *>(a.workspace + (int64_t)(tile.y + row) * RP + c));
        *reinterpret_cast<float4 *>(&sh.h[row][c]) = v;
      }
      __syncthreads();
      if (!Half2<T>::kBf16) {
        for (int row = warp; row < kTile; row += kWarps) {
          const int e = row_exponent<RP>(sh.h[row]);
          __syncwarp();
          for (int c = lane; c < RP; c += 32) sh.h[row][c] = ldexpf(sh.h[row][c], e);
          if (lane == 0) sh.unscale[row] = ldexpf(1.0f, -e);
        }
        __syncthreads();
      }
      make_fragments<T, RP, 4, kTerms, kStride>(&sh.h[0][0], sh.frag);
    }
    __syncthreads();

    // ---- the old outputs ahead of their use
    Cursor cy(blk0, per), c(blk0, per);
    int y_blk = blk0, y_m = 0, y_slot = 0, at_slot = 0;
    auto fetch = [&]() {
      if (y_blk < blocks) {
        const int col = cy.i * 32 + q * 8;
        const char *y = static_cast<const char *>(a.y[cy.p]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int t = sh.token[y_m * 16 + r * 8 + g];
          const bool valid = t >= 0 && col < O;
          const char *from = valid ? y + (t * a.ldy + col) * kSize : y;
#pragma unroll
          for (int i = 0; i < kWords; ++i)
            cp_async16(smem_u32(ring + ((y_slot * 2 + r) * kWords + i) * 32), from + 16 * i * valid, valid);
        }
        if (++y_m == 4) {
          y_m = 0, y_blk += step;
          cy.next(step, per);
        }
      }
      y_slot = y_slot + 1 == kAhead ? 0 : y_slot + 1;
      cp_async_commit();
    };
    for (int i = 0; i < kAhead - 1; ++i) fetch();

    uint4 w[4][RP == 16 ? 1 : KS / 2];
    auto load_b = [&](const Cursor &at) {
      const uint16_t *b = static_cast<const uint16_t *>(a.b[at.p]) + ((int64_t)id * O + at.i * 32) * a.R;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = (g >> 1) * 8 + 2 * j + (g & 1);
        const bool in = at.i * 32 + r < O;
        const uint16_t *row = b + r * a.R;
        if (RP == 16) {
          const uint2 v = in && q * 4 < a.R ? __ldg(reinterpret_cast<const uint2 *>(row + q * 4)) : make_uint2(0, 0);
          w[j][0].x = v.x, w[j][0].y = v.y;
        } else {
#pragma unroll
          for (int s = 0; s < KS / 2; ++s)
            w[j][s] = in && s * 32 + q * 8 < a.R ? __ldg(reinterpret_cast<const uint4 *>(row + s * 32 + q * 8)) : make_uint4(0, 0, 0, 0);
        }
      }
    };
    if (id >= 0 && blk0 < blocks) load_b(c);
    for (int blk = blk0; blk < blocks; blk += step) {
      const int p = c.p, col = c.i * 32 + q * 8;
      c.next(step, per);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        float d[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.0f;
        if (id >= 0) {
#pragma unroll
          for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int i = 0; i < kTerms; ++i) {
              const uint4 f = sh.frag[i][m][s][lane];
              const uint32_t hf[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint4 b = w[j][RP == 16 ? 0 : s / 2];
                mma16816<T>(d[j], hf, s % 2 ? b.z : b.x, s % 2 ? b.w : b.y);
              }
            }
          if (m == 3 && blk + step < blocks) load_b(c);
        }
        cp_async_wait<kAhead - 2>();
        uint4 y[2][kWords];
#pragma unroll
        for (int i = 0; i < 2 * kWords; ++i) y[i / kWords][i % kWords] = ring[(at_slot * 2 * kWords + i) * 32];
        at_slot = at_slot + 1 == kAhead ? 0 : at_slot + 1;
        fetch();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int t = sh.token[m * 16 + r * 8 + g];
          if (id >= 0) {
            const float f = Half2<T>::kBf16 ? 1.0f : sh.unscale[m * 16 + r * 8 + g];
            float add[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) add[2 * j] = d[j][2 * r] * f, add[2 * j + 1] = d[j][2 * r + 1] * f;
            if (OUT32) {
              y[r][0] = add_floats(y[r][0], add);
              y[r][kWords - 1] = add_floats(y[r][kWords - 1], add + 4);
            } else {
              y[r][0] = out_bf16 ? add_pairs<__nv_bfloat16>(y[r][0], add) : add_pairs<__half>(y[r][0], add);
            }
          }
          if (t >= 0 && col < O) {
            uint4 *to = reinterpret_cast<uint4 *>(static_cast<char *>(a.out[p]) + (t * a.ldo + col) * kSize);
#pragma unroll
            for (int i = 0; i < kWords; ++i) to[i] = y[r][i];
          }
        }
      }
    }
    cp_async_wait<0>();
  }
}

template <typename K, typename... Args>
int launch_one(K kern, int64_t grid, size_t smem, int C, cudaStream_t s, const Args &...args) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return cuda_error(e, "adapter launch");
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)grid);
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
  cfg.numAttrs = C > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) return cuda_error(e, "adapter launch");
  note_launch();
  return TP_OK;
}

template <typename T, int RP>
int launch(const LoraArgs &a, cudaStream_t s) {
  int64_t tiles = a.T / kTile + a.most;  // at most
  if (tiles > (1 << 20)) tiles = 1 << 20;
  const int64_t slots = 2 * sm_count();
  int C = 1;
  while (C < 8 && tiles * C * 2 <= slots) C *= 2;
  if (int rc = launch_one(lora_shrink_kernel<T, RP>, tiles * C, sizeof(ShrinkShared<RP>), C, s, a, C)) return rc;
  const int64_t blocks = (a.O + 31) / 32 * a.ny, most = (blocks + kWarps - 1) / kWarps;
  int64_t S = (4 * slots + tiles - 1) / tiles;
  S = S < 1 ? 1 : S < most ? S : most;
  if (a.out_dt == TP_F32)
    return launch_one(lora_expand_kernel<T, RP, true>, tiles * S, sizeof(ExpandShared<T, RP, true>), 1, s, a, (int)S);
  return launch_one(lora_expand_kernel<T, RP, false>, tiles * S, sizeof(ExpandShared<T, RP, false>), 1, s, a, (int)S);
}

template <typename T>
int launch(const LoraArgs &a, int RP, cudaStream_t s) {
  switch (RP) {
    case 16: return launch<T, 16>(a, s);
    case 32: return launch<T, 32>(a, s);
    case 64: return launch<T, 64>(a, s);
    default: return launch<T, 128>(a, s);
  }
}

}  // namespace

int launch_lora_prompt(const LoraArgs &a, int RP, cudaStream_t s) {
  return a.dt == TP_BF16 ? launch<__nv_bfloat16>(a, RP, s) : launch<__half>(a, RP, s);
}

}  // namespace tp
