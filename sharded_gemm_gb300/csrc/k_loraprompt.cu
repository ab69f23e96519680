// k_loraprompt.cu -- the adapters of k_lora.cu for steps of many tokens, as two passes:
//   h[i] = sum_p x_p[t] A_p[a]^T   for the token t at place i of the plan,
//   out_r[t] = y_r[t] + (scale_a h[i]) B_r[a]^T,
// h float32 in the call's workspace.  A tile is up to 64 tokens of one adapter, in the second
// pass 128.
//
// Bound by bytes: the tokens' rows once, the outputs' once in and once out, an adapter once a
// tile from L2.  So both passes are streams whose loads run ahead: each lane copies what it
// alone will read into its part of a ring in shared memory (16-byte asynchronous copies), with
// no barrier between the copy and its use.  (As one kernel, h exchanged within a cluster, the
// barriers between the products stood in the way of the streams, and registers for both were
// too many: 309 us for 8192 tokens, R = 64, 4096 x 11008, where 66 us of bytes move.)
//
// Measured: those 107 us, the first pass 27 (67 MB) and the second 83 (361 MB, 4.4 TB/s: the
// products of h's two terms; one alone took 70); 5003 tokens, R = 16, 11008 x 4096, float32
// outputs 62, passes of 25 (110 MB) and 32 (164 MB).
#include "lora.cuh"

namespace tp {
namespace {

constexpr int kShrinkTile = 64;  // tokens of a tile of the first pass

// The tiles of a plan (in all lanes).
__device__ __forceinline__ int count_tiles(const LoraArgs &a, int groups, int rows, bool none) {
  int n = 0;
#pragma unroll 4
  for (int base = 0; base < groups; base += 32)
    n += (int)__reduce_add_sync(0xffffffffu, tiles_of(a, group_at(a, base + threadIdx.x % 32, groups), rows, none));
  return n;
}

// Into how many shares of `units` to split each tile's work (1..most, at most 32) for a grid
// of CTAs: the least turns times what a share takes, `start` units' time and its own.
__device__ __forceinline__ int shares_of(int tiles, int grid, int units, int start, int most) {
  const int s = threadIdx.x % 32 + 1;
  const unsigned turns = ((unsigned)(tiles * s) + grid - 1) / (unsigned)grid;  // tiles: 2^25 at most
  const unsigned cost = s <= most ? min(turns * ((unsigned)start + (unsigned)(units + s - 1) / (unsigned)s), 0x3ffffffu) : 0x3ffffffu;
  return (int)(__reduce_min_sync(0xffffffffu, cost << 5 | (unsigned)(s - 1)) & 31) + 1;
}
// The first pass's shares of the contraction, the same in both: kG warps take a unit each.
template <int RP>
__device__ __forceinline__ int splits_of(const LoraArgs &a, int tiles, int grid);

// ---------------------------------------------------------------- the first pass
// Eight warps: kM groups of MW blocks of 16 tokens, kG stretches of the contraction.  A ring
// holds units of 32 elements of the contraction: the tokens' rows, then the adapter's.  Of a
// tile of few tokens only the blocks that hold one are read and multiplied, and one group takes
// it if that holds it all (1100 tokens of 250 adapters, R = 16, 4096 x 4096, both passes: 134 us
// with all four blocks, 61 without, 56 so, 59 with what has come since).  A tile's contraction may
// be split over several CTAs, whose sums lie side by side in the workspace until the second pass
// adds them, in their order.
template <int RP>
struct ShrinkShared {
  static constexpr int MW = RP == 128 ? 2 : RP == 64 ? 4 : 2, kM = 4 / MW, kG = kWarps / kM, kStride = RP + 4;
  static constexpr int kAhead = RP == 128 ? 2 : RP == 16 ? 4 : 3, kRows = 2 * MW + RP / 8;  // pieces of 512 bytes a unit
  static constexpr int kCtas = RP <= 32 ? 2 : 1;                                            // of an SM
  union {
    uint4 ring[kWarps][kAhead][kRows][32];
    float part[kG * kShrinkTile][kStride];  // the groups' of a tile's rows, or of its first half
  };
  int token[kShrinkTile];
};
template <int RP>
__device__ __forceinline__ int splits_of(const LoraArgs &a, int tiles, int sms) {
  typedef ShrinkShared<RP> Shared;
  const int units = (int)((a.K + 31) / 32) * a.nx;
  return shares_of(tiles, Shared::kCtas * sms, (units + Shared::kG - 1) / Shared::kG, 6, a.splits);
}

template <typename T, int RP>
__global__ void __launch_bounds__(kLoraThreads, ShrinkShared<RP>::kCtas)
    lora_shrink_kernel(const __grid_constant__ LoraArgs a, int sms) {
  typedef ShrinkShared<RP> Shared;
  constexpr int NT = RP / 8, MW = Shared::MW, kAhead = Shared::kAhead, kStride = Shared::kStride;
  extern __shared__ __align__(16) uint8_t smem[];
  Shared &sh = *reinterpret_cast<Shared *>(smem);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, q = lane % 4;
  const int K = (int)a.K, per = (K + 31) / 32, units = per * a.nx;
  griddep_launch_dependents();
  griddep_wait();
  const int groups = groups_of(a), tiles = count_tiles(a, groups, kShrinkTile, false);
  const unsigned S = splits_of<RP>(a, tiles, sms);
  int base = 0;
  int64_t before = 0;
  int4 tile;
  for (unsigned item = blockIdx.x; item < (unsigned)(tiles * S); item += gridDim.x) {
    if (!find_tile(a, groups, kShrinkTile, false, item / S, base, before, tile)) break;
    // the split's units (of 2^25 and a few at most) in turn to the groups of warps: neighbours
    // read a row's neighbouring bytes
    const int M = tile.z <= MW * 16 ? 1 : Shared::kM, G = kWarps / M, m0 = warp % M * MW, rows = M * MW * 16;
    const int id = tile.x, split = item % S, u0 = (int)((unsigned)(units * split) / S) + warp / M;
    const int u1 = (int)((unsigned)(units * (split + 1)) / S);
    __syncthreads();  // the last item's sums are read
    read_tokens(a, tile, kShrinkTile, sh.token);
    __syncthreads();
    const int used = (tile.z + 15) / 16 - m0;  // the warp's blocks of 16 tokens that have one
    int64_t row[2 * MW];  // where the lane's rows of x begin; without a token, any: its h is not kept
#pragma unroll
    for (int i = 0; i < 2 * MW; ++i) row[i] = max(sh.token[(m0 + i / 2) * 16 + i % 2 * 8 + g], 0) * a.ldx;
    Cursor c(u0, per);
    int ahead = u0, x_slot = 0, slot_at = 0;
    const uint16_t *x[2 * MW], *w = nullptr;
    auto part = [&]() {
#pragma unroll
      for (int i = 0; i < 2 * MW; ++i) x[i] = static_cast<const uint16_t *>(a.x[c.p]) + row[i];
      w = static_cast<const uint16_t *>(a.a[c.p]) + ((int64_t)id * a.R + g) * K;
    };
    if (u0 < u1) part();
    auto fetch = [&]() {
      if (ahead < u1) {
        // behind the rows' end zeros, and in place of the rows that the adapter lacks
        const int at = c.i * 32 + q * 8, k = at < K ? at : 0, size = at < K ? 16 : 0;
        const uint32_t to = smem_u32(&sh.ring[warp][x_slot][0][lane]);
#pragma unroll
        for (int i = 0; i < 2 * MW; ++i)
          if (i / 2 < used) cp_async16(to + i * 512, x[i] + k, size);
        const uint16_t *from = w + k;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const bool in = j * 8 + g < a.R;
          cp_async16(to + (2 * MW + j) * 512, in ? from : w, in ? size : 0);
          from += 8 * (int64_t)K;
        }
        const int p = c.p;
        c.next(G, per);
        if (c.p != p && ahead + G < u1) part();
      }
      ahead += G;
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
    for (int u = u0; u < u1; u += G) {
      cp_async_wait<kAhead - 2>();
      const uint4(*const ring)[32] = sh.ring[warp][slot_at];
      uint32_t f[MW][2][4];  // put together once: the products want them in neighbouring registers
#pragma unroll
      for (int m = 0; m < MW; ++m) {
        const uint4 r0 = ring[2 * m][lane], r1 = ring[2 * m + 1][lane];
        keep4(f[m][0], r0.x, r1.x, r0.y, r1.y);
        keep4(f[m][1], r0.z, r1.z, r0.w, r1.w);
      }
      fetch();
      constexpr int JW = 4 / MW;  // four products between two of one sum
#pragma unroll
      for (int j = 0; j < NT; j += JW) {
        uint4 v[JW];
#pragma unroll
        for (int k = 0; k < JW; ++k) v[k] = ring[2 * MW + j + k][lane];
#pragma unroll
        for (int k = 0; k < JW; ++k)
#pragma unroll
          for (int m = 0; m < MW; ++m)
            if (m < used) mma16816<T>(acc[m][j + k], f[m][0], v[k].x, v[k].y);
#pragma unroll
        for (int k = 0; k < JW; ++k)
#pragma unroll
          for (int m = 0; m < MW; ++m)
            if (m < used) mma16816<T>(acc[m][j + k], f[m][1], v[k].z, v[k].w);
      }
      slot_at = slot_at + 1 == kAhead ? 0 : slot_at + 1;
    }
    cp_async_wait<0>();
    __syncthreads();  // the rings are read
#pragma unroll
    for (int m = 0; m < MW; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float *to = &sh.part[warp / M * rows + (m0 + m) * 16 + g][j * 8 + q * 2];
        *reinterpret_cast<float2 *>(to) = make_float2(acc[m][j][0], acc[m][j][1]);
        *reinterpret_cast<float2 *>(to + 8 * kStride) = make_float2(acc[m][j][2], acc[m][j][3]);
      }
    __syncthreads();
    float *const to = a.workspace + ((int64_t)split * a.T + tile.y) * RP;
    for (int i = tid; i < tile.z * (RP / 4); i += kLoraThreads) {
      const int r = i / (RP / 4), col = i % (RP / 4) * 4;
      float4 sum = *reinterpret_cast<const float4 *>(&sh.part[r][col]);
      for (int j = 1; j < G; ++j) sum = add4(sum, *reinterpret_cast<const float4 *>(&sh.part[j * rows + r][col]));
      *reinterpret_cast<float4 *>(to + (int64_t)r * RP + col) = sum;
    }
  }
}

// ---------------------------------------------------------------- the second pass
// A warp takes 32 columns of a tile at a time, its lane 8 of them in the rows g and g + 8 of
// each block of 16 tokens.  Old values are fetched into the place that was just read, four
// blocks ahead.  The adapter's rows are read once a tile, from L2, whose rate bounds the pass
// with the outputs: so its tiles are as long as its shared memory allows for two CTAs an SM.
template <typename T, int RP, typename O>
struct ExpandShared {
  static constexpr bool OUT32 = sizeof(O) == 4;
  static constexpr int kTerms = terms<T>(OUT32);
  static constexpr int kStride = RP + 4, kWords = OUT32 ? 2 : 1, kTile = RP == 128 ? 64 : 128;  // tokens
  union {
    uint4 ring[kWarps][4][2 * kWords][32];
    float h[kTile][kStride];
  };
  uint4 b[kWarps][RP == 16 ? 4 : RP / 8][32];  // the adapter's rows
  uint4 frag[kTerms][kTile / 16][RP / 16][32];
  int64_t y_row[kTile], out_row[kTile];  // where the rows begin, in bytes; out: without a token, -1
  int token[kTile];
  float unscale[kTile];
};

__device__ __forceinline__ uint4 add_floats(uint4 y, const float *d) {
  return make_uint4(__float_as_uint(__uint_as_float(y.x) + d[0]), __float_as_uint(__uint_as_float(y.y) + d[1]),
                    __float_as_uint(__uint_as_float(y.z) + d[2]), __float_as_uint(__uint_as_float(y.w) + d[3]));
}
template <typename O>
__device__ __forceinline__ uint4 pack8(const float *d) {
  return make_uint4(Half2<O>::pack(d[0], d[1]), Half2<O>::pack(d[2], d[3]), Half2<O>::pack(d[4], d[5]),
                    Half2<O>::pack(d[6], d[7]));
}
template <typename O>
__device__ __forceinline__ void unpack8(const uint4 &v, float *d) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Half2<O>::unpack(w[i]);
    d[2 * i] = f.x, d[2 * i + 1] = f.y;
  }
}

// O: the outputs' type.
template <typename T, int RP, typename O>
__global__ void __launch_bounds__(kLoraThreads, RP == 128 ? 1 : 2)
    lora_expand_kernel(const __grid_constant__ LoraArgs a, int sms) {
  typedef ExpandShared<T, RP, O> Shared;
  constexpr bool OUT32 = Shared::OUT32;
  constexpr int KS = RP / 16, kTerms = Shared::kTerms, kStride = Shared::kStride, kWords = Shared::kWords;
  constexpr int kTile = Shared::kTile;
  // 16-bit outputs: the products are added to the old values, whose sums lose less than the
  // rounding does; float32 ones keep the old values out of the products' sums
  constexpr bool kSeed = !OUT32 && Half2<T>::kBf16;
  extern __shared__ __align__(16) uint8_t smem[];
  Shared &sh = *reinterpret_cast<Shared *>(smem);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, q = lane % 4;
  const int cols = (int)a.O, per = (cols + 31) / 32, blocks = per * a.ny;
  uint4 *const ring = &sh.ring[warp][0][0][lane];
  griddep_launch_dependents();
  // The plan too is read behind it: what kernels wrote before is promised there alone.  (Read ahead,
  // under the first pass's end, it saved 2 us.)
  griddep_wait();
  const int groups = groups_of(a), with = count_tiles(a, groups, kShrinkTile, false), splits = splits_of<RP>(a, with, sms);
  const int tiles = count_tiles(a, groups, kTile, !a.in_place);
  const unsigned S = shares_of(tiles, gridDim.x, (blocks + kWarps - 1) / kWarps, 3, 32);
  const int step = S * kWarps;
  int base = 0;
  int64_t before = 0;
  int4 tile;
  for (unsigned item = blockIdx.x; item < (unsigned)(tiles * S); item += gridDim.x) {
    if (!find_tile(a, groups, kTile, !a.in_place, item / S, base, before, tile)) break;
    const int id = tile.x, blk0 = item % S * kWarps + warp;
    __syncthreads();
    read_tokens(a, tile, kTile, sh.token);
    if (tid < kTile) {  // read_tokens' own thread
      const int t = sh.token[tid];
      sh.y_row[tid] = max(t, 0) * a.ldy * (int64_t)sizeof(O);
      sh.out_row[tid] = t < 0 ? -1 : t * a.ldo * (int64_t)sizeof(O);
    }
    if (id >= 0) {
      const float scale = a.scales ? __ldg(a.scales + id) : 1.0f;
      for (int i = tid; i < kTile * RP / 4; i += kLoraThreads) {
        const int r = i / (RP / 4), c = i % (RP / 4) * 4;
        float4 v = make_float4(0, 0, 0, 0);
        if (r < tile.z)
          for (int k = 0; k < splits; ++k)
            v = add4(v, __ldcg(reinterpret_cast<const float4 *>(a.workspace + ((int64_t)k * a.T + tile.y + r) * RP + c)));
        *reinterpret_cast<float4 *>(&sh.h[r][c]) = scaled_h(v, scale, c, a.R);
      }
      __syncthreads();
      if (!Half2<T>::kBf16) {
        for (int r = warp; r < kTile; r += kWarps) {
          const int e = row_exponent<RP>(sh.h[r]);
          __syncwarp();
          for (int c = lane; c < RP; c += 32) sh.h[r][c] = ldexpf(sh.h[r][c], e);
          if (lane == 0) sh.unscale[r] = ldexpf(1.0f, -e);
        }
        __syncthreads();
      }
      make_fragments<T, RP, kTile / 16, kTerms, kStride>(&sh.h[0][0], sh.frag);
    }
    __syncthreads();

    const int mc = (tile.z + 15) / 16;  // blocks of 16 tokens
    Cursor cy(blk0, per), c(blk0, per);
    int y_blk = blk0, y_m = 0, y_slot = 0;
    // the old values that cy and y_m name, four blocks of 16 tokens ahead of their use
    auto fetch = [&]() {
      if (y_blk < blocks) {
        const char *y = static_cast<const char *>(a.y[cy.p]);
        int at[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          const int col = cy.i * 32 + lane_col(OUT32, i, q);
          at[i] = (col < cols ? col : 0) * (int)sizeof(O);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < kWords; ++i)
            cp_async16(smem_u32(ring + ((y_slot * 2 + r) * kWords + i) * 32), y + sh.y_row[y_m * 16 + r * 8 + g] + at[i], 16);
        if (++y_m == mc) {
          y_m = 0, y_blk += step;
          cy.next(step, per);
        }
      }
      y_slot = (y_slot + 1) & 3;
      cp_async_commit();
    };
    // the adapter's rows of the columns that c names
    constexpr int kB = RP == 16 ? 1 : KS / 2;
    auto fetch_b = [&]() {
      const uint16_t *b = static_cast<const uint16_t *>(a.b[c.p]) + ((int64_t)id * cols + c.i * 32) * a.R;
      const uint32_t to = smem_u32(&sh.b[warp][0][lane]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = b_row(OUT32, j, g);
        const bool in = c.i * 32 + r < cols;
#pragma unroll
        for (int s = 0; s < kB; ++s) {
          const int k = RP == 16 ? q * 4 : s * 32 + q * 8;
          const bool valid = in && k < a.R;
          if (RP == 16) cp_async8(to + j * 512, valid ? b + r * a.R + k : b, valid ? 8 : 0);
          else cp_async16(to + (j * kB + s) * 512, valid ? b + r * a.R + k : b, valid ? 16 : 0);
        }
      }
    };
    if (id >= 0 && blk0 < blocks) fetch_b();
#pragma unroll
    for (int m = 0; m < 4; ++m) fetch();
    int slot = 0;
    for (int blk = blk0; blk < blocks; blk += step) {
      const int col = c.i * 32 + lane_col(OUT32, 0, q);
      char *const out = static_cast<char *>(a.out[c.p]) + col * (int)sizeof(O);
      c.next(step, per);
      uint4 w[4][kB];
      if (id >= 0) {
        // they came with the old values of the first block of 16 tokens, mc copies ago
        if (mc < 4) cp_async_wait<0>(); else cp_async_wait<3>();
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int s = 0; s < kB; ++s) w[j][s] = sh.b[warp][j * kB + s][lane];
      }
#pragma unroll 2
      for (int m = 0; m < mc; ++m) {
        uint4 y[2][kWords];
        float d[4][4], add[2][8];
        auto take = [&]() {
          cp_async_wait<3>();
#pragma unroll
          for (int i = 0; i < 2 * kWords; ++i) y[i / kWords][i % kWords] = ring[(slot * 2 * kWords + i) * 32];
        };
        if (kSeed) {
          take();
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            unpack8<typename std::conditional<OUT32, __half, O>::type>(y[r][0], add[r]);
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j][2 * r] = add[r][2 * j], d[j][2 * r + 1] = add[r][2 * j + 1];
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.0f;
        }
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
          if (m == 0 && blk + step < blocks) fetch_b();  // the products have read the rows
        }
        if (!kSeed) take();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float f = Half2<T>::kBf16 || id < 0 ? 1.0f : sh.unscale[m * 16 + r * 8 + g];
#pragma unroll
          for (int j = 0; j < 4; ++j) add[r][2 * j] = d[j][2 * r] * f, add[r][2 * j + 1] = d[j][2 * r + 1] * f;
          if constexpr (OUT32) {
            if (id >= 0) y[r][0] = add_floats(y[r][0], add[r]), y[r][1] = add_floats(y[r][1], add[r] + 4);
          } else if constexpr (kSeed) {
            if (id >= 0) y[r][0] = pack8<O>(add[r]);
          } else if (id >= 0) {
            float old[8];
            unpack8<O>(y[r][0], old);
#pragma unroll
            for (int i = 0; i < 8; ++i) add[r][i] += old[i];
            y[r][0] = pack8<O>(add[r]);
          }
          const int64_t row = sh.out_row[m * 16 + r * 8 + g];
          if (row >= 0) {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
              if (col + i * 16 < cols) *reinterpret_cast<uint4 *>(out + row + i * 64) = y[r][i];
          }
        }
        fetch();  // into the place of the values just used
        slot = (slot + 1) & 3;
      }
    }
    cp_async_wait<0>();
  }
}

template <typename K>
int launch_one(K kern, int ctas, size_t smem, const LoraArgs &a, cudaStream_t s) {
  const int sms = sm_count();
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) e = launch_pdl(kern, dim3((unsigned)(ctas * sms)), dim3(kLoraThreads), smem, s, a, sms);
  if (e != cudaSuccess) return cuda_error(e, "adapter launch");
  note_launch();
  return TP_OK;
}

template <typename T, int RP, typename O>
int launch_expand(const LoraArgs &a, cudaStream_t s) {
  return launch_one(lora_expand_kernel<T, RP, O>, RP == 128 ? 1 : 2, sizeof(ExpandShared<T, RP, O>), a, s);
}

template <typename T, int RP>
int launch(const LoraArgs &a, cudaStream_t s) {
  if (int rc = launch_one(lora_shrink_kernel<T, RP>, ShrinkShared<RP>::kCtas, sizeof(ShrinkShared<RP>), a, s)) return rc;
  if (a.out_dt == TP_F32) return launch_expand<T, RP, float>(a, s);
  return a.out_dt == TP_F16 ? launch_expand<T, RP, __half>(a, s) : launch_expand<T, RP, __nv_bfloat16>(a, s);
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
