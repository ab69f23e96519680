// k_pprefill.cu -- tp_paged_prefill on the tensor cores: attention of ragged
// chunks of tokens over the paged cache.
//
// A unit is one sequence, rank, key-value head, group of its query heads and
// block of tokens: two query tiles of 128 rows, a row being one (token, head),
// so all query heads of a key-value head share its key and value tiles.  Per
// key tile of 128 positions and query tile,
//   S = Q K^T          128 x 128, float32 in tensor memory
//   P = 2^(S' - m)     S' the scaled (and capped) scores in log2, m the row's
//                      running maximum; rounded to the 16-bit type, over S
//   O += P V           128 x D, float32 in tensor memory, P read from there
// One thread owns one row, so maxima and sums need no exchange.  O is rescaled
// only where a row's maximum grows by more than 2^8 (the 16-bit terms and the
// float32 sums have room for that), which after the first tiles is rare.
//
// Persistent, one CTA per SM, twelve warps:
//   warp 0       units (dealt out at run time: their lengths differ) and the
//                tensor copies of the key and value pages, 128-byte swizzled,
//                into a ring of tiles;
//   warp 1       one thread issues every tcgen05.mma: P0 V, Q0 K', P1 V, Q1 K',
//                so one query tile's softmax runs under the other's products;
//   warps 2, 3   the next unit's queries into shared memory;
//   warps 4..11  softmax, rescale and output, one warpgroup per query tile.
// Where whole units would leave SMs idle (a few tokens over a long cache) every CTA
// takes an equal range of the list of all units' key tiles.  A unit that several CTAs
// hold leaves each one's O, m and l in the workspace, and the last warp to come joins its
// rows, in CTA order.  One token over 16384 positions, 32 heads on 8: 167 us whole, 37 so;
// 64 over 32768: 331, 78; 512 over 8192: 96, 65; 2048 over 16384: 335, 317.
// Rows of a value tile behind the sequence's end (or in pages that are not
// read) are written as zeros: stale rows never meet a product.  A value within the
// sequence that is not finite does, with the terms 0 of rows that do not see it:
// their sums are NaN, which is noticed, and these rows are computed again (redo_rows).
//
// Tensor rate bounds long chunks: 4 D flop per visible pair.  Of it, what holds
// the kernel back is shared memory: Q K^T reads both operands from there, 128
// bytes a cycle, which is all there is.  Measured: 8192 tokens, 32 heads of 128,
// causal, 371 to 387 us a call in a graph of 20 and 393 to 410 in a long run (1350 to 1480
// TFLOP/s, 70 to 77% of cuBLAS's burst rate); 2 x 1024 tokens over 4000..8192 cached positions,
// 32 heads on 8, 175 and 186 us; five prompts of 7..150 tokens 14 us.
#include "attn.cuh"
#include "mma16.cuh"
#include "ptx.cuh"

namespace tp {
namespace {

constexpr int kThreads = 384;
constexpr int kTile = 128;  // rows of a query tile, positions of a key tile
constexpr float kSlack = 8.0f;
constexpr int kUnitTiles = 2;  // what a unit costs besides its tiles, in tiles (1.6 to 1.9 us at D = 128)
constexpr int kJoinTiles = 6;  // and what a CTA's two shared ones cost more
// Registers a thread: 384 * 168 at launch = 128 * 88 + 256 * 208.
constexpr int kRegsFew = 88, kRegsMany = 208;

template <int D>
struct Sh {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kHalf = kTile * 128;  // bytes of a tile's 64-value column block
  static constexpr int kQBytes = 2 * kTileBytes;
  static constexpr int kSlots = D == 128 ? 5 : 10;
  static constexpr int kSmem = kQBytes + kSlots * kTileBytes + 1024;
};

template <int MAXN>
struct PrefillArgs {
  CUtensorMap k[MAXN], v[MAXN];
  AttnArgs a;
  int groups, gsize, tpt;  // head groups of a key-value head, heads of a group, tokens of a query tile
  int box;                 // rows of a page copy
  int vec_q, vec_o;
  int *counters;  // units dealt, CTAs at the end; with few units, of every CTA's shared one, parts come by warp
  float *ws;      // parts of shared units: of a CTA two, of those each query tile's D + 2 values of 128 rows
  int few;        // so few units that their tiles may be shared
  uint64_t wait_ns;
};

struct Unit {
  int valid, b, r, h, grp;
  int tok0, ntok;  // first token (row of q), tokens
  int pos0;        // its position
  int to, prefix;  // positions of the sequence; bidirectional ones
  int seen0;       // no row of the unit sees a position below this
  int j0;          // first key tile's position
  int n[2];        // key tiles of the query tiles
  // where the unit's key tiles are shared with other CTAs:
  int shared, c0, others;  // the first of them, how many besides this one
};

// A CTA's range in the list of all units' key tiles, and the unit it has come to.
struct Walk {
  long long x0, x1, share;  // from, to, of every CTA; in tiles, each unit counted kUnitTiles more
  long long at;             // where the unit begins
  int64_t b, t0;
  int tokens, to, prefix;   // of sequence b
  int blocks, rank, hu, n;  // its blocks, the unit's place among them and among the heads, its tiles
  int ranged;
};

struct Control {
  uint64_t unit_full[2], unit_free[2], q_full[2], q_free[2], s_full[2], p_full[2][2], o_done[2], drain;
  uint64_t kv_full[10], kv_free[10];
  Unit unit[2];
  Walk walk;
  uint32_t tmem;
  int abort;
};

// mbar_wait without its out-of-line slow path: a call would spill the scores
// that the softmax warps hold in registers.
__device__ __forceinline__ bool wait_inline(uint32_t bar, uint32_t parity, uint64_t limit_ns, int *status,
                                            volatile int *abort) {
  bool done = mbar_try_wait(bar, parity);
  if (!__all_sync(0xffffffffu, done)) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1; !done; ++i) {
      done = mbar_try_wait(bar, parity);
      if (done || (i & 31)) continue;
      if (*abort) break;
      if (globaltimer_ns() - t0 > limit_ns) {
        atomicMin(status, TP_ERR_TIMEOUT);
        *abort = 1;
      }
    }
    done = __all_sync(0xffffffffu, done);
  }
  return done;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// The n lowest bits, n clamped to 0..32.
__device__ __forceinline__ uint32_t low_bits(int n) {
  n = n < 0 ? 0 : n > 32 ? 32 : n;
  return (uint32_t)((1ull << n) - 1);
}
// Two float32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t y;
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ void unpack2(uint64_t x, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t y;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
  return y;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t y;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
  return y;
}

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The tokens of sequence b, kept inside q whatever cu_seqlens holds.
__device__ __forceinline__ void token_range(const AttnArgs &a, int64_t b, int64_t &t0, int64_t &t1) {
  const int64_t c0 = a.cu_seqlens[b], c1 = a.cu_seqlens[b + 1];
  t0 = c0 < 0 ? 0 : c0 > a.T ? a.T : c0;
  t1 = c1 < t0 ? t0 : c1 > a.T ? a.T : c1;
  if (c0 != t0 || c1 != t1) record_bad_value(a.status);
}

// Outputs of a warp's rows again (those of the lanes set in `rows`, of one sequence and key-value
// head), on the CUDA cores, each from the positions that it sees alone.  Four rows at a time: a lane
// has their scores with one of 32 positions, and every 32nd of their values.  A row is known by its
// output's address, and all else found again from that: the softmax warps, whose registers are full,
// would have to keep it (2 x 1024 tokens over 4000..8192 took 179 us so, 175 as it is, 173 without any
// of this).  Rare, and slow: 512 tokens over 65536 positions, 8 heads of 128, take 0.14 ms and with a
// last value that is not finite 278.
template <typename T, int D>
__device__ __noinline__ void redo_rows(const AttnArgs &a, bool vec_q, uint32_t rows, T *out) {
  constexpr int E = D / 32, R = 4;
  const int lane = threadIdx.x % 32, first = __ffs(rows) - 1;
  // the rank whose output the rows are in (the ranks' may be column blocks of one matrix), token and head
  int r = 0, hq = 0;
  int64_t tok = 0;
  for (; r < a.N; ++r) {
    const int64_t off = out - static_cast<const T *>(a.o[r]);
    tok = off / a.ldo;
    const int64_t col = off - tok * a.ldo;
    hq = (int)(col / D);
    if (__shfl_sync(0xffffffffu, off >= 0 && tok < a.T && col < (int64_t)a.Hq * D, first)) break;
  }
  if (r == a.N) return;
  const T *k_cache = static_cast<const T *>(a.k_cache[r]), *v_cache = static_cast<const T *>(a.v_cache[r]);
  const int h = __shfl_sync(0xffffffffu, hq, first) / (a.Hq / a.Hk);
  int64_t b = 0;  // the last sequence whose first token is not behind the rows'
  for (int64_t top = a.B, t0 = __shfl_sync(0xffffffffu, tok, first); top - b > 1;) {
    const int64_t mid = (b + top) / 2;
    if (a.cu_seqlens[mid] <= t0) b = mid; else top = mid;
  }
  // the lane's row sees [lo, hi) and [0, prefix)
  const int64_t len = a.seq_lens[b], n = len < 0 ? 0 : len > a.cap ? a.cap : len;
  const int64_t pos = n - a.cu_seqlens[b + 1] + tok, pre = a.prefix_lens ? a.prefix_lens[b] : 0;
  const int prefix = (int)(pre < 0 ? 0 : pre > n ? n : pre);
  const int lo = (int)(a.window && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0), hi = (int)(pos + 1 < n ? pos + 1 : n);
  const uint16_t *q = static_cast<const uint16_t *>(a.q[r]) + tok * a.ldq + (int64_t)hq * D;
  for (int f0 = 0; f0 < 32; f0 += R) {
    const uint32_t some = rows >> f0 & ((1u << R) - 1);
    if (!some) continue;
    const bool mine = rows >> lane & 1 && lane / R == f0 / R;
    const int from = (int)__reduce_min_sync(0xffffffffu, mine ? (prefix > 0 ? 0 : lo) : 0x7fffffff) & ~31;
    const int end = __reduce_max_sync(0xffffffffu, mine ? max(hi, prefix) : 0);
    const uint16_t *qr[R];
    float m[R], l[R], acc[R][E];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      qr[i] = reinterpret_cast<const uint16_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(q), f0 + i));
      m[i] = -INFINITY, l[i] = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[i][e] = 0.0f;
    }
#pragma unroll 1
    for (int j0 = from; j0 < end; j0 += 32) {
      const int j = j0 + lane;
      int64_t row = -1;
      if (j < end) {
        const int pg = a.block_table[b * a.ld_table + (j >> a.page_log2)];
        if (pg >= 0 && pg < a.pages) row = pg * a.ld_page + ((int64_t)h * a.page + (j & (a.page - 1))) * D;
      }
      float p[R];
#pragma unroll
      for (int i = 0; i < R; ++i) p[i] = 0.0f;
      if (row >= 0) {
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 x = *reinterpret_cast<const uint4 *>(k_cache + row + c * 8);
          const uint32_t k[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < R; ++i) {
            if (!(some >> i & 1)) continue;
            uint32_t qq[4];
            if (vec_q) {
              const uint4 y = __ldg(reinterpret_cast<const uint4 *>(qr[i] + c * 8));
              qq[0] = y.x, qq[1] = y.y, qq[2] = y.z, qq[3] = y.w;
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                qq[e] = (uint32_t)__ldg(qr[i] + c * 8 + 2 * e) | (uint32_t)__ldg(qr[i] + c * 8 + 2 * e + 1) << 16;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 kf = Half2<T>::unpack(k[e]), qf = Half2<T>::unpack(qq[e]);
              p[i] = fmaf(qf.x, kf.x, fmaf(qf.y, kf.y, p[i]));
            }
          }
        }
      }
      uint32_t seen[R], any = 0;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int lo_i = __shfl_sync(0xffffffffu, lo, f0 + i), hi_i = __shfl_sync(0xffffffffu, hi, f0 + i);
        const float log2e = 1.4426950408889634f;
        const bool is = row >= 0 && (some >> i & 1) && ((j >= lo_i && j < hi_i) || j < prefix);
        seen[i] = __ballot_sync(0xffffffffu, is);
        any |= seen[i];
        float s = a.softcap > 0.0f ? capped(p[i] * (2.0f * log2e * a.scale / a.softcap), a.softcap * log2e)
                                   : p[i] * (a.scale * log2e);
        if (!is) s = -INFINITY;
        float top = s, sum;
#pragma unroll
        for (int x = 16; x > 0; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        top = fmaxf(top, m[i]);
        const float to = top == -INFINITY ? 0.0f : top, keep = exp2_approx(m[i] - to);
        m[i] = top;
        sum = p[i] = exp2_approx(s - to);
#pragma unroll
        for (int x = 16; x > 0; x /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        l[i] = fmaf(l[i], keep, sum);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[i][e] *= keep;
      }
      if (!any) continue;
#pragma unroll 1
      for (int x0 = 0; x0 < 32; x0 += 8) {
        // eight positions' values at a time, loaded whether seen or not (position 0 of page 0 where
        // there is no page), and used where seen
        T v[8][E];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int64_t at = __shfl_sync(0xffffffffu, row < 0 ? 0 : row, x0 + x);
#pragma unroll
          for (int e = 0; e < E; ++e) v[x][e] = v_cache[at + lane + 32 * e];
        }
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const float pi = __shfl_sync(0xffffffffu, p[i], x0 + x);
            const bool is = seen[i] >> (x0 + x) & 1;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[i][e] = is ? fmaf(pi, static_cast<float>(v[x][e]), acc[i][e]) : acc[i][e];
          }
      }
      bool lost = true;  // nothing behind this changes the rows any more
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) lost = lost && (isnan(acc[i][e]) || !(some >> i & 1));
      if (__all_sync(0xffffffffu, lost)) break;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      T *o = reinterpret_cast<T *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out), f0 + i));
      const float inv = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
      if (some >> i & 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) o[lane + 32 * e] = static_cast<T>(acc[i][e] * inv);
      }
    }
  }
}

template <typename T, int D, int MAXN>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ PrefillArgs<MAXN> pa) {
  using S = Sh<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Control ctl;
  const AttnArgs &a = pa.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t smem = (smem_u32(smem_raw) + 1023) & ~1023u;
  uint8_t *smem_gen = smem_raw + (smem - smem_u32(smem_raw));
  const uint32_t q_smem = smem, kv_smem = smem + S::kQBytes;
  volatile int *abort = &ctl.abort;
  const uint64_t limit = pa.wait_ns;
  // the same answer in every lane of the warp
  auto wait = [&](uint64_t &bar, uint32_t parity) {
    return (bool)__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), parity, limit, a.status, abort));
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctl.unit_full[i]), 1);
      mbar_init(smem_u32(&ctl.unit_free[i]), 11);  // warps 1..11
      mbar_init(smem_u32(&ctl.q_full[i]), 64);
      mbar_init(smem_u32(&ctl.q_free[i]), 1);
      mbar_init(smem_u32(&ctl.s_full[i]), 1);
      mbar_init(smem_u32(&ctl.p_full[i][0]), 4);
      mbar_init(smem_u32(&ctl.p_full[i][1]), 4);
      mbar_init(smem_u32(&ctl.o_done[i]), 1);
    }
    mbar_init(smem_u32(&ctl.drain), 1);
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(smem_u32(&ctl.kv_full[i]), 1);
      mbar_init(smem_u32(&ctl.kv_free[i]), 1);
    }
    ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl.tmem), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's, so they begin at the first
  griddep_launch_dependents();
  griddep_wait();

  const int block = 2 * pa.tpt;  // tokens of a unit
  const int heads_units = a.N * a.Hk * pa.groups;

  if (warp < 4) {
    regs_down<kRegsFew>();
    if (warp == 0) {
      // ---------------------------------------------------------------- units, keys and values
      int64_t cur_b = 0;
      long long cur_base = 0;  // units of the sequences before cur_b
      long long u = blockIdx.x;
      int slot = 0, seq = 0;
      unsigned fills = 0;  // ring slots filled so far
      uint32_t kv_phase = 0;
      bool ok = true;
      Walk &wk = ctl.walk;
      // a sequence's length and bidirectional part, inside what the table can hold
      auto lengths = [&](int64_t b, int &to, int &prefix) {
        int64_t n = a.seq_lens[b];
        if (n < 0 || n > a.cap) {
          record_bad_value(a.status);
          n = n < 0 ? 0 : a.cap;
        }
        to = (int)n;
        const int pre = a.prefix_lens ? a.prefix_lens[b] : 0;
        prefix = pre < 0 ? 0 : pre > to ? to : pre;
      };
      // the first position that a block whose first is pos0 may see
      auto seen_from = [&](int pos0, int prefix) {
        const int lo = a.window && prefix == 0 ? pos0 - a.window + 1 : 0;
        return lo < 0 ? 0 : lo;
      };
      // key tiles of block qb of a sequence
      auto tiles_of = [&](int tokens, int to, int prefix, int qb) {
        const int pos0 = to - tokens + qb * block;
        int hi = tokens - qb * block < block ? to : pos0 + block;
        if (hi < prefix) hi = prefix;
        const int j0 = seen_from(pos0, prefix) & ~(kTile - 1);
        return hi > j0 ? (hi - j0 + kTile - 1) / kTile : 0;
      };
      wk.ranged = 0;
      if (pa.few) {
        // Few units: their lengths, and whether equal ranges of tiles are likely to end before whole
        // units would.  (Ranges are not shorter than an eighth of the longest unit: all its
        // parts are read back by one CTA.  An eighth over the even share and a join are allowed
        // for: 2 x 1024 tokens over 4000..8192 took 182 us in ranges, 177 whole.)
        auto cost_of = [&](int64_t b, long long &units, int &longest) {
          int64_t t0 = 0, t1 = 0;
          int to, prefix;
          long long sum = 0;
          if (b >= a.B) return sum;
          token_range(a, b, t0, t1);
          lengths(b, to, prefix);
          const int blocks = (int)((t1 - t0 + block - 1) / block);
          for (int qb = 0; qb < blocks; ++qb) {
            const int n = tiles_of((int)(t1 - t0), to, prefix, qb);
            sum += kUnitTiles + n;
            longest = n > longest ? n : longest;
          }
          units += (long long)blocks * heads_units;
          return sum * heads_units;
        };
        long long total = 0, units = 0;
        int longest = 0;
        for (int64_t b = lane; b < a.B + lane; b += 32) total += cost_of(b, units, longest);
#pragma unroll
        for (int m = 16; m > 0; m /= 2) {
          total += __shfl_xor_sync(0xffffffffu, total, m);
          units += __shfl_xor_sync(0xffffffffu, units, m);
          longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, m));
        }
        const long long even = (total + gridDim.x - 1) / gridDim.x;
        const int least = max(4, (longest + 7) / 8);
        const long long share = even > least ? even : least;
        // whole units: the longest, or as many turns as it takes of average ones
        const long long turns = (units + gridDim.x - 1) / gridDim.x;
        const long long whole = turns <= 1 ? longest + kUnitTiles : turns * total / units;
        if (whole > share + share / 8 + kJoinTiles) {
          const long long x0 = blockIdx.x * share < total ? blockIdx.x * share : total;
          // the sequence that holds x0
          long long base = 0;
          int64_t b = a.B;
          for (int64_t b32 = 0; b32 < a.B; b32 += 32) {
            const long long mine = cost_of(b32 + lane, units, longest);
            long long run = mine;
#pragma unroll
            for (int m = 1; m < 32; m *= 2) {
              const long long o = __shfl_up_sync(0xffffffffu, run, m);
              if (lane >= m) run += o;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, base + run > x0);
            if (hit) {
              const int l = __ffs(hit) - 1;
              b = b32 + l;
              base += __shfl_sync(0xffffffffu, run - mine, l);
              break;
            }
            base += __shfl_sync(0xffffffffu, run, 31);
          }
          if (lane == 0) {
            wk.ranged = 1;
            wk.share = share;
            wk.x0 = x0;
            wk.x1 = x0 + share < total ? x0 + share : total;
            wk.at = base;
            wk.b = b - 1;
            wk.blocks = wk.rank = wk.n = 0;
            wk.hu = heads_units - 1;
          }
        }
      }
      __syncwarp();
      // the walk's next unit (lane 0)
      auto step = [&](bool begin) {
        if (!begin) wk.at += kUnitTiles + wk.n;
        if (++wk.hu < heads_units) return;
        wk.hu = 0;
        if (++wk.rank >= wk.blocks) {
          wk.rank = 0;
          do {
            if (++wk.b >= a.B) return;
            int64_t t0, t1;
            token_range(a, wk.b, t0, t1);
            wk.t0 = t0;
            wk.tokens = (int)(t1 - t0);
            wk.blocks = (wk.tokens + block - 1) / block;
          } while (wk.blocks == 0);
          lengths(wk.b, wk.to, wk.prefix);
        }
        wk.n = tiles_of(wk.tokens, wk.to, wk.prefix, wk.blocks - 1 - wk.rank);
      };
      if (lane == 0 && wk.ranged) {
        step(true);
        // to the block, and the head, that hold x0
        while (wk.b < a.B && wk.at + (long long)heads_units * (kUnitTiles + wk.n) <= wk.x0) {
          wk.at += (long long)heads_units * (kUnitTiles + wk.n);
          ++wk.rank;
          wk.n = tiles_of(wk.tokens, wk.to, wk.prefix, wk.blocks - 1 - wk.rank);
        }
        if (wk.b < a.B) {
          wk.hu = (int)((wk.x0 - wk.at) / (kUnitTiles + wk.n));
          wk.at += (long long)wk.hu * (kUnitTiles + wk.n);
        }
      }
      __syncwarp();
      for (;; ++seq) {
        int64_t b = -1, t0 = 0;
        int tokens = 0, qb = 0, hu = 0, from = 0, to_tile = 0x7fffffff;
        Unit w;
        w.shared = 0;
        if (wk.ranged) {
          // the next unit of which a tile is in the range, or that has none and begins in it
          if (lane == 0) {
            for (; wk.b < a.B && wk.at < wk.x1; step(false)) {
              const long long f = wk.at + kUnitTiles;
              const long long lo = wk.x0 > f ? wk.x0 - f : 0, hi = wk.x1 - f < wk.n ? wk.x1 - f : wk.n;
              if (wk.n == 0 ? wk.at < wk.x0 : hi <= lo) continue;
              b = wk.b, t0 = wk.t0, tokens = wk.tokens;
              qb = wk.blocks - 1 - wk.rank, hu = wk.hu;
              from = (int)lo, to_tile = wk.n ? (int)hi : 0;
              if (to_tile - from < wk.n) {
                w.shared = 1;
                w.c0 = (int)(f / wk.share);
                w.others = (int)((f + wk.n - 1) / wk.share) - w.c0;
              }
              step(false);
              break;
            }
          }
          b = __shfl_sync(0xffffffffu, b, 0);
          t0 = __shfl_sync(0xffffffffu, t0, 0);
          tokens = __shfl_sync(0xffffffffu, tokens, 0);
          qb = __shfl_sync(0xffffffffu, qb, 0);
          hu = __shfl_sync(0xffffffffu, hu, 0);
          from = __shfl_sync(0xffffffffu, from, 0);
          to_tile = __shfl_sync(0xffffffffu, to_tile, 0);
        } else {
          // find unit u: 32 sequences at a time from the cursor
          while (cur_b < a.B) {
            int64_t x0 = 0, x1 = 0;
            if (cur_b + lane < a.B) token_range(a, cur_b + lane, x0, x1);
            long long mine = (x1 - x0 + block - 1) / block * heads_units, run = mine;
#pragma unroll
            for (int m = 1; m < 32; m *= 2) {
              const long long o = __shfl_up_sync(0xffffffffu, run, m);
              if (lane >= m) run += o;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, cur_base + run > u);
            if (hit) {
              const int l = __ffs(hit) - 1;
              b = cur_b + l;
              const long long local = u - (cur_base + __shfl_sync(0xffffffffu, run - mine, l));
              t0 = __shfl_sync(0xffffffffu, x0, l);
              tokens = (int)(__shfl_sync(0xffffffffu, x1, l) - t0);
              // longest first, a block's heads side by side: the CTAs then walk the
              // same key tiles of a head at about the same time
              hu = (int)(local % heads_units);
              qb = (tokens + block - 1) / block - 1 - (int)(local / heads_units);
              break;
            }
            cur_base += __shfl_sync(0xffffffffu, run, 31);
            cur_b += 32;
          }
        }
        w.valid = b >= 0;
        if (w.valid) {
          w.b = (int)b;
          w.grp = hu % pa.groups;
          w.h = hu / pa.groups % a.Hk;
          w.r = hu / pa.groups / a.Hk;
          w.tok0 = (int)t0 + qb * block;
          w.ntok = tokens - qb * block < block ? tokens - qb * block : block;
          lengths(b, w.to, w.prefix);
          w.pos0 = w.to - tokens + qb * block;
          w.seen0 = seen_from(w.pos0, w.prefix);
          w.j0 = w.seen0 & ~(kTile - 1);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int rows = w.ntok - i * pa.tpt < pa.tpt ? w.ntok - i * pa.tpt : pa.tpt;
            int hi = w.pos0 + i * pa.tpt + rows;  // behind the last row's position
            if (hi < w.prefix) hi = w.prefix;
            if (hi > w.to) hi = w.to;
            const int n = rows > 0 && hi > w.j0 ? (hi - w.j0 + kTile - 1) / kTile : 0;
            w.n[i] = n < from ? 0 : (n < to_tile ? n : to_tile) - from;  // of the part
          }
          w.j0 += from * kTile;
        }
        const int us = seq & 1;
        if (seq >= 2) ok = wait(ctl.unit_free[us], ((seq >> 1) - 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          ctl.unit[us] = w;
          mbar_arrive(smem_u32(&ctl.unit_full[us]));
        }
        if (!w.valid) {
          if (lane == 0 && !wk.ranged) {
            // out of units: the last CTA to see that clears the counters for the next call
            // (every CTA's additions to the first are done before its one to the second)
            __threadfence();
            if (atomicAdd(pa.counters + 1, 1) == (int)gridDim.x - 1) {
              __threadfence();
              atomicExch(pa.counters, 0);
              atomicExch(pa.counters + 1, 0);
            }
          }
          break;
        }
        const int nmax = w.n[0] > w.n[1] ? w.n[0] : w.n[1];
        const int *table = a.block_table + w.b * a.ld_table;
        const int pieces = kTile / pa.box;  // page copies of a tile
        // lane i < pieces: the row in the map of piece i of tile j, -1 where it is not read
        auto lookup = [&](int j) {
          const int pj = w.j0 + j * kTile + lane * pa.box;
          if (lane >= pieces || pj >= w.to || pj + pa.box <= w.seen0) return -1;
          const int pg = table[pj >> a.page_log2];
          if (pg < 0 || pg >= a.pages) {
            record_bad_value(a.status);
            return -1;
          }
          return (int)(pg * (a.ld_page / D) + (int64_t)w.h * a.page + (pj & (a.page - 1)));
        };
        int next_row = nmax > 0 ? lookup(0) : -1;
        for (int j = 0; j < nmax && ok; ++j) {
          const int jt = w.j0 + j * kTile, row = next_row;
          const bool part = jt + (lane + 1) * pa.box > w.to;
          const uint32_t read = __ballot_sync(0xffffffffu, row >= 0);
          const uint32_t whole = __ballot_sync(0xffffffffu, row >= 0 && !part);
          if (j + 1 < nmax) next_row = lookup(j + 1);  // a tile ahead: the table's latency stays off the copies
          for (int kv = 0; kv < 2 && ok; ++kv) {
            ok = wait(ctl.kv_free[slot], kv_phase ^ 1);
            if (!ok) break;
            const uint32_t dst = kv_smem + slot * S::kTileBytes;
            const uint32_t bar = smem_u32(&ctl.kv_full[slot]);
            const uint32_t copied = kv ? whole : read;  // hidden keys may hold anything, values not
            if (kv && whole != (pieces == 32 ? 0xffffffffu : (1u << pieces) - 1)) {
              // rows of the pieces that are not copied whole: the sequence's own, and zeros
              uint8_t *gen = smem_gen + S::kQBytes + slot * S::kTileBytes;
              for (int p = 0; p < pieces; ++p) {
                if (whole >> p & 1) continue;
                const int prow = __shfl_sync(0xffffffffu, row, p), pj = jt + p * pa.box;
                const T *src = static_cast<const T *>(a.v_cache[w.r]) + (int64_t)prow * D;
                for (int e = lane; e < pa.box * (D / 8); e += 32) {
                  const int i = e / (D / 8), c = e % (D / 8), tr = p * pa.box + i;
                  uint4 x = make_uint4(0, 0, 0, 0);
                  if (prow >= 0 && pj + i < w.to) x = *reinterpret_cast<const uint4 *>(src + (int64_t)i * D + c * 8);
                  *reinterpret_cast<uint4 *>(gen + (c >> 3) * S::kHalf + tr * 128 + (((c & 7) ^ (tr & 7)) << 4)) = x;
                }
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
            if (lane == 0) mbar_arrive_expect_tx(bar, __popc(copied) * pa.box * D * 2);
            __syncwarp();
            if (copied >> lane & 1) {
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_2d(dst + c * S::kHalf + lane * pa.box * 128, kv ? &pa.v[w.r] : &pa.k[w.r], bar, c * 64, row);
            }
            if (++slot == S::kSlots) slot = 0, kv_phase ^= 1;
            ++fills;
          }
        }
        if (!ok) break;
        // The next unit is asked for only now, a ring of tiles before this one's
        // products end: asked for earlier, units went to CTAs that were still busy.
        if (!wk.ranged) {
          if (lane == 0) u = (long long)gridDim.x + atomicAdd(pa.counters, 1);
          u = __shfl_sync(0xffffffffu, u, 0);
        }
      }
      if (!ok) {
        // gave up: the copies in flight still land in this CTA's shared memory
        for (unsigned i = 0; i < S::kSlots && i < fills; ++i) {
          const unsigned f = fills - 1 - i;
          mbar_wait(smem_u32(&ctl.kv_full[f % S::kSlots]), (f / S::kSlots) & 1, limit, a.status, nullptr);
        }
        __syncwarp();
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- products
      // elect_one in place of a branch on the lane: the compiler then keeps the
      // descriptors in uniform registers (an MMA runs for 64 cycles; issued from
      // a plain branch it took 95).
      if (elect_one()) {
        auto wait1 = [&](uint64_t &bar, uint32_t parity) {
          return mbar_wait(smem_u32(&bar), parity, limit, a.status, abort);
        };
        constexpr uint32_t fmt = Half2<T>::kBf16 ? 1 : 0;
        constexpr uint32_t id_qk = umma_idesc_f16(fmt, 0, kTile, kTile), id_pv = umma_idesc_f16(fmt, 1, kTile, D);
        int slot = 0, n0 = 0, n1 = 0;
        uint32_t kv_phase = 0, p_phase0 = 0, p_phase1 = 0, q_phase = 0;
        bool ok = true;
        auto qk = [&](int i, int ks) {  // S_i = Q_i K^T, K in ring slot ks
          tc_fence_after();
          const uint32_t qa = q_smem + i * S::kTileBytes, kb = kv_smem + ks * S::kTileBytes;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk / 4) * S::kHalf + (kk % 4) * 32;
            umma_f16(tmem + i * kTile, umma_desc_sw128(qa + off, 16, 1024), umma_desc_sw128(kb + off, 16, 1024), id_qk,
                     kk > 0);
          }
          umma_commit(smem_u32(&ctl.s_full[i]));
        };
        auto pv = [&](int i, int vs, bool add, int half) {  // O_i (+)= P_i V over half the positions, V in slot vs
          tc_fence_after();
          const uint32_t vb = kv_smem + vs * S::kTileBytes;
#pragma unroll
          for (int k = 0; k < kTile / 32; ++k) {
            const int kk = half * (kTile / 32) + k;
            umma_f16_ts(tmem + 256 + i * D, tmem + i * kTile + kk * 8, umma_desc_sw128(vb + kk * 2048, S::kHalf, 1024),
                        id_pv, add || kk > 0);
          }
          if (half) umma_commit(smem_u32(&ctl.o_done[i]));
        };
        auto take = [&](int &taken) {  // the next filled ring slot
          taken = slot;
          ok = wait1(ctl.kv_full[slot], kv_phase);
          if (++slot == S::kSlots) slot = 0, kv_phase ^= 1;
        };
        auto first = [&](int i, int n, int ks) {
          if (ok) ok = wait1(ctl.q_full[i], q_phase);  // loaded for every unit, used or not
          if (!ok) return;
          if (n > 0) qk(i, ks);
          if (n <= 1) umma_commit(smem_u32(&ctl.q_free[i]));
        };
        auto values = [&](int i, int n, int j, int vs, uint32_t &p_phase) {
          if (!ok || j >= n) return;
          ok = wait1(ctl.p_full[i][0], p_phase);
          if (!ok) return;
          pv(i, vs, j > 0, 0);
          ok = wait1(ctl.p_full[i][1], p_phase);
          if (!ok) return;
          p_phase ^= 1;
          pv(i, vs, true, 1);
        };
        auto scores = [&](int i, int n, int j, int ks) {
          if (!ok) return;
          if (j + 1 < n) qk(i, ks);
          if (j + 2 == n) umma_commit(smem_u32(&ctl.q_free[i]));
        };
        for (int seq = 0; ok; ++seq) {
          const int us = seq & 1;
          ok = wait1(ctl.unit_full[us], (seq >> 1) & 1);
          if (!ok) break;
          const int valid = ctl.unit[us].valid;
          n0 = ctl.unit[us].n[0], n1 = ctl.unit[us].n[1];
          mbar_arrive(smem_u32(&ctl.unit_free[us]));
          if (!valid) break;
          const int nmax = n0 > n1 ? n0 : n1;
          int ks = 0, vs = 0, next_vs = 0;
          if (nmax > 0) take(ks);
          first(0, n0, ks);
          first(1, n1, ks);
          q_phase ^= 1;
          if (nmax > 0 && ok) {
            umma_commit(smem_u32(&ctl.kv_free[ks]));
            take(vs);
          }
          // Waits stand where products just issued still run.
          for (int j = 0; j < nmax && ok; ++j) {
            values(0, n0, j, vs, p_phase0);
            if (ok && j + 1 < nmax) take(ks);
            scores(0, n0, j, ks);
            if (ok && j + 1 < nmax) take(next_vs);
            values(1, n1, j, vs, p_phase1);
            scores(1, n1, j, ks);
            if (!ok) break;
            umma_commit(smem_u32(&ctl.kv_free[vs]));
            if (j + 1 < nmax) umma_commit(smem_u32(&ctl.kv_free[ks]));
            vs = next_vs;
          }
        }
        // every product issued has ended before the tensor memory goes back
        umma_commit(smem_u32(&ctl.drain));
        mbar_wait(smem_u32(&ctl.drain), 0, limit, a.status, nullptr);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------------- queries
      const int th = threadIdx.x - 64, G = a.Hq / a.Hk;
      const int row0 = th / (D / 8), tk0 = row0 / pa.gsize, hd0 = row0 - tk0 * pa.gsize;
      const int step_tk = 64 / (D / 8) / pa.gsize, step_hd = 64 / (D / 8) - step_tk * pa.gsize;
      const int64_t step_src = step_tk * a.ldq + (int64_t)step_hd * D, wrap_src = a.ldq - (int64_t)pa.gsize * D;
      for (int seq = 0;; ++seq) {
        const int us = seq & 1;
        if (!wait(ctl.unit_full[us], (seq >> 1) & 1)) break;
        const Unit w = ctl.unit[us];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl.unit_free[us]));
        if (!w.valid) {
          // rows of no sequence are zero
          int64_t c0 = a.cu_seqlens[0], c1 = a.cu_seqlens[a.B];
          c0 = c0 < 0 ? 0 : c0 > a.T ? a.T : c0;
          c1 = c1 < c0 ? c0 : c1 > a.T ? a.T : c1;
          const int64_t outside = c0 + a.T - c1, row = (int64_t)a.Hq * D;
          for (int64_t i = blockIdx.x * 64 + th; i < outside * a.N * row; i += (int64_t)gridDim.x * 64) {
            const int64_t t = i / row % outside;
            const int r = (int)(i / row / outside);
            static_cast<T *>(a.o[r])[(t < c0 ? t : c1 + t - c0) * a.ldo + i % row] = static_cast<T>(0.0f);
          }
          break;
        }
        const int heads = G - w.grp * pa.gsize < pa.gsize ? G - w.grp * pa.gsize : pa.gsize;
        const T *q = static_cast<const T *>(a.q[w.r]) + (int64_t)w.tok0 * a.ldq +
                     ((int64_t)w.h * G + w.grp * pa.gsize) * D;
        bool ok = true;
        for (int i = 0; i < 2; ++i) {
          if (seq > 0) ok = wait(ctl.q_free[i], (seq - 1) & 1);
          if (!ok) break;
          // this thread's column of 8 values, in every kStep-th row; the row's token and head
          // go along without divisions (with them a unit's queries took 2 us longer)
          constexpr int kStep = 64 / (D / 8);
          const int c = th % (D / 8);
          const uint32_t base = i * S::kTileBytes + (c >> 3) * S::kHalf;
          const int tokens = w.ntok - i * pa.tpt < pa.tpt ? w.ntok - i * pa.tpt : pa.tpt;
          int tk = tk0, hd = hd0;
          const T *src = q + (int64_t)(i * pa.tpt + tk) * a.ldq + (int64_t)hd * D + c * 8;
#pragma unroll 4
          for (int row = th / (D / 8); row < kTile; row += kStep) {
            const bool live = tk < tokens && hd < heads;
            const uint32_t off = base + row * 128 + (((c & 7) ^ (row & 7)) << 4);
            if (pa.vec_q) {
              cp_async16(q_smem + off, live ? src : q, live);
            } else {
              uint16_t x[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) x[k] = live ? reinterpret_cast<const uint16_t *>(src)[k] : 0;
              *reinterpret_cast<uint4 *>(smem_gen + off) =
                  make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
            }
            tk += step_tk, hd += step_hd, src += step_src;
            if (hd >= pa.gsize) hd -= pa.gsize, ++tk, src += wrap_src;
          }
          cp_async_commit();
          cp_async_wait<0>();
          fence_proxy_async_smem();
          mbar_arrive(smem_u32(&ctl.q_full[i]));
        }
        if (!ok) break;
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax and output
    regs_up<kRegsMany>();
    const int i = (warp - 4) / 4, row = (warp % 4) * 32 + lane, G = a.Hq / a.Hk;
    const uint32_t lanes = (uint32_t)(warp % 4) << 21;  // lane 32 * (warp % 4) of tensor memory
    const uint32_t s_tmem = tmem + i * kTile + lanes, o_tmem = tmem + 256 + i * D + lanes;
    const int tk = row / pa.gsize, hd = row - tk * pa.gsize;
    const bool cap = a.softcap > 0.0f;
    const float log2e = 1.4426950408889634f;
    // log2 scores: s * scale * log2e, or with a cap c: c * log2e * tanh(s * scale / c),
    // from 2 s * scale / c * log2e by capped()
    const float scale = cap ? 2.0f * log2e * a.scale / a.softcap : a.scale * log2e;
    const float cap2 = a.softcap * log2e;
    uint32_t s_phase = 0, o_count = 0;
    bool ok = true;
    for (int seq = 0;; ++seq) {
      const int us = seq & 1;
      if (!wait_inline(smem_u32(&ctl.unit_full[us]), (seq >> 1) & 1, limit, a.status, abort)) break;
      const Unit w = ctl.unit[us];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl.unit_free[us]));
      if (!w.valid) break;
      const int heads = G - w.grp * pa.gsize < pa.gsize ? G - w.grp * pa.gsize : pa.gsize;
      const bool live = tk < pa.tpt && i * pa.tpt + tk < w.ntok && hd < heads;
      T *out = live ? static_cast<T *>(a.o[w.r]) + (int64_t)(w.tok0 + i * pa.tpt + tk) * a.ldo +
                          ((int64_t)w.h * G + w.grp * pa.gsize + hd) * D
                    : nullptr;
      const int tiles = w.n[i], prefix = w.prefix;
      int jt = w.j0;
      // this row sees [lo, hi) and [0, prefix)
      const int pos = w.pos0 + i * pa.tpt + tk;
      const int hi = pos + 1 < w.to ? pos + 1 : w.to;
      const int lo = a.window && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
      // what every row of the tile sees
      const int t_last = (w.ntok - i * pa.tpt < pa.tpt ? w.ntok - i * pa.tpt : pa.tpt) - 1;
      const int all_hi = w.pos0 + i * pa.tpt + 1 < w.to ? w.pos0 + i * pa.tpt + 1 : w.to;
      const int pos_last = w.pos0 + i * pa.tpt + t_last;
      const int all_lo = a.window && pos_last - a.window + 1 > 0 ? pos_last - a.window + 1 : 0;
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < tiles; ++j, jt += kTile) {
        ok = wait_inline(smem_u32(&ctl.s_full[i]), s_phase, limit, a.status, abort);
        s_phase ^= 1;
        if (!ok) break;
        tc_fence_after();
        float s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_tmem + c * 32, s[c]);
        tmem_wait_ld();
        if (cap) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int x = 0; x < 32; ++x)
              s[c][x] = capped(s[c][x] * scale, cap2);
        }
        if (!(jt + kTile <= prefix || (jt >= all_lo && jt + kTile <= all_hi))) {
          // one bit a position: compared one by one they cost the registers of the scores
          const int from = lo - jt, to = hi - jt, pre = prefix - jt;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t seen = (low_bits(to - c * 32) & ~low_bits(from - c * 32)) | low_bits(pre - c * 32);
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (!(seen >> x & 1)) s[c][x] = -INFINITY;
          }
        }
        const float f = cap ? 1.0f : scale;
        const uint64_t f2 = pack2(f, f);
        // terms of half the positions into tensor memory, and their sum
        auto half = [&](int h, float neg) {
          const uint64_t neg2 = pack2(neg, neg);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int c = 2 * h; c < 2 * h + 2; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              float e0, e1;
              unpack2(fma2(pack2(s[c][2 * x], s[c][2 * x + 1]), f2, neg2), e0, e1);
              e0 = exp2_approx(e0), e1 = exp2_approx(e1);
              sum[x & 1] = add2(sum[x & 1], pack2(e0, e1));
              pk[x] = Half2<T>::pack(e0, e1);
            }
            tmem_st16(s_tmem + c * 16, pk);
          }
          float a0, a1;
          unpack2(add2(sum[0], sum[1]), a0, a1);
          return a0 + a1;
        };
        auto ready = [&](int h) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl.p_full[i][h]));
        };
        // The first half goes by the maximum so far while the tile's own is
        // found: most tiles do not raise it, and the two run side by side.
        float sum0 = half(0, m == -INFINITY ? 0.0f : -m);
        float top[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          top[c] = fmaxf(s[c][0], s[c][1]);
#pragma unroll
          for (int x = 2; x < 32; x += 2) top[c] = max3(top[c], s[c][x], s[c][x + 1]);
        }
        const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * f;
        const bool rise = mx > m + kSlack;
        if (__any_sync(0xffffffffu, rise)) {
          const float keep = rise ? exp2_approx(m - mx) : 1.0f;
          if (rise) m = mx;
          l *= keep;
          if (j > 0) {
            // the products up to the previous tile have to be in O
            ok = wait_inline(smem_u32(&ctl.o_done[i]), (o_count - 1) & 1, limit, a.status, abort);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              float o[16];
              uint32_t r[16];
              tmem_ld16(o_tmem + c * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 16; ++x) r[x] = __float_as_uint(o[x] * keep);
              tmem_st16(o_tmem + c * 16, r);
            }
          }
          sum0 = half(0, m == -INFINITY ? 0.0f : -m);
        }
        ready(0);
        l += sum0 + half(1, m == -INFINITY ? 0.0f : -m);
        ready(1);
        ++o_count;
      }
      if (!ok) break;
      if (tiles > 0) {
        ok = wait_inline(smem_u32(&ctl.o_done[i]), (o_count - 1) & 1, limit, a.status, abort);
        if (!ok) break;
        tc_fence_after();
      }
      auto sums = [&](int c, float (&o)[32]) {  // this row's O, 32 values of it
        if (tiles > 0) {
          tmem_ld32(o_tmem + c * 32, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = 0.0f;
        }
      };
      // the part left by CTA c, from a row on: value x at x * kTile
      auto part = [&](int c, int of) {
        return pa.ws + (size_t)((c * 2 + (c == w.c0)) * 2 + i) * ((D + 2) * kTile) + of;
      };
      auto factor = [](float mc, float to) { return mc == -INFINITY ? 0.0f : exp2_approx(mc - to); };
      bool joins = false;
      // In a join of few rows, the first `rows` of the warp (8 or 16), several lanes share a
      // row's values: lane g * rows + r has values of row r.
      int rows = 32, g = 0, jrow = row;
      bool mine_too = live;  // this lane has values to join
      float top = m;
      if (w.shared) {
        float *mine = part(blockIdx.x, row);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          sums(c, o);
          if (live) {
#pragma unroll
            for (int x = 0; x < 32; ++x) mine[(c * 32 + x) * kTile] = o[x];
          }
          __syncwarp();
        }
        if (live) mine[D * kTile] = m, mine[(D + 1) * kTile] = l;
        __syncwarp();
        int came = 0;
        if (lane == 0) {
          // releases the warp's rows, and acquires those of the CTAs counted before
          int *count = pa.counters + 2 + w.c0 * 8 + (warp - 4);
          asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(came) : "l"(count) : "memory");
          if (came == w.others) *count = 0;  // ready for the next call
        }
        joins = __shfl_sync(0xffffffffu, came, 0) == w.others;
        __syncwarp();  // what lane 0 has acquired, for the other lanes: the shuffle orders no memory
        if (!joins) {
          tc_fence_before();
          continue;
        }
        const uint32_t alive = __ballot_sync(0xffffffffu, live);
        rows = alive >> 8 == 0 ? 8 : alive >> 16 == 0 ? 16 : 32;
        g = lane / rows;
        const int from = lane % rows;
        jrow = row - lane + from;
        mine_too = alive >> from & 1;
        out = reinterpret_cast<T *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out), from));
        const int end = mine_too ? w.c0 + w.others + 1 : 0;
        float sum = 0.0f;
        top = -INFINITY;
        for (int c0 = w.c0; c0 < end; c0 += 4) {
          float mc[4], lc[4], mx = top;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            mc[k] = c0 + k < end ? __ldcg(part(c0 + k, jrow) + D * kTile) : -INFINITY;
            lc[k] = c0 + k < end ? __ldcg(part(c0 + k, jrow) + (D + 1) * kTile) : 0.0f;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) mx = fmaxf(mx, mc[k]);
          sum *= factor(top, mx);
          top = mx;
#pragma unroll
          for (int k = 0; k < 4; ++k) sum = fmaf(factor(mc[k], top), lc[k], sum);
        }
        l = sum;
      }
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      bool nan = false;
#pragma unroll 1
      for (int c0 = 0; c0 < D / 32; c0 += 32 / rows) {
        const int c = c0 + g;
        float o[32];
        if (!joins) {
          sums(c, o);
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = 0.0f;
          // in CTA order, so that who came last changes no rounding; two parts' loads at a time
          float own[32];
          sums(c0, own);
          // (its own part too is read back where lanes share rows)
          const int end = mine_too && c < D / 32 ? w.c0 + w.others + 1 : 0, me = rows == 32 ? (int)blockIdx.x : -1;
          for (int k0 = w.c0; k0 < end; k0 += 2) {
            float v[2][32], f[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const bool is = k0 + k < end && k0 + k != me;
              const float *p = part(is ? k0 + k : w.c0, jrow);
              f[k] = k0 + k == me ? m : is ? __ldcg(p + D * kTile) : -INFINITY;
#pragma unroll
              for (int x = 0; x < 32; ++x) v[k][x] = is ? __ldcg(p + (c * 32 + x) * kTile) : own[x];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float e = factor(f[k], top);
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = fmaf(e, v[k][x], o[x]);
            }
          }
        }
        if (out && c < D / 32) {
          uint32_t pk[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) pk[x] = Half2<T>::pack(o[2 * x] * inv, o[2 * x + 1] * inv);
          auto as2 = [](const uint32_t &u) { return *reinterpret_cast<const typename Half2<T>::Pair *>(&u); };
          auto top2 = as2(pk[0]), low2 = as2(pk[1]);
#pragma unroll
          for (int x = 2; x < 16; x += 2) top2 = __hmax2_nan(top2, as2(pk[x])), low2 = __hmax2_nan(low2, as2(pk[x + 1]));
          top2 = __hmax2_nan(top2, low2);
          nan |= __hisnan(top2.x) || __hisnan(top2.y);
          if (pa.vec_o) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              *reinterpret_cast<uint4 *>(out + c * 32 + x * 8) =
                  make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
          } else {
            uint16_t *p = reinterpret_cast<uint16_t *>(out + c * 32);
#pragma unroll
            for (int x = 0; x < 16; ++x) p[2 * x] = (uint16_t)pk[x], p[2 * x + 1] = (uint16_t)(pk[x] >> 16);
          }
        }
        __syncwarp();
      }
      // A value of the tile that is not finite gives NaN in rows that do not see it as well (0 times
      // it): rows whose scores are numbers and whose sums are not are taken again.  (The check costs
      // 1 us of 173, packed and with the maximum that keeps NaN; a chain of compares, 3.)
      uint32_t redo = __ballot_sync(0xffffffffu, nan && !isnan(inv));
      if (redo) {
        if (rows <= 16) redo |= redo >> 16;
        if (rows == 8) redo |= redo >> 8;
        redo_rows<T, D>(a, pa.vec_q, rows < 32 ? redo & ((1u << rows) - 1) : redo, out);
        __syncwarp();
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(ctl.tmem, 512);
  }
}

template <typename T, int D, int MAXN>
int launch(const AttnArgs &a, cudaStream_t s) {
  PrefillArgs<MAXN> p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  const int G = a.Hq / a.Hk;
  p.groups = (G + kTile - 1) / kTile;
  p.gsize = (G + p.groups - 1) / p.groups;
  p.tpt = kTile / p.gsize;
  p.box = a.page < kTile ? a.page : kTile;
  p.wait_ns = wait_limit_ns();
  p.vec_q = (a.ldq * 2) % 16 == 0;
  p.vec_o = (a.ldo * 2) % 16 == 0;
  const CUtensorMapDataType mt = Half2<T>::kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  for (int r = 0; r < a.N; ++r) {
    p.vec_q = p.vec_q && (uintptr_t)a.q[r] % 16 == 0;
    p.vec_o = p.vec_o && (uintptr_t)a.o[r] % 16 == 0;
    const uint64_t rows = (uint64_t)a.pages * (uint64_t)(a.ld_page / D);
    if (rows > 0x7fffffff) return set_error(TP_ERR_UNSUPPORTED, "a cache of more than 2^31 - 1 rows of D");
    // without pages nothing is read, but a map needs an address
    const void *kc = a.pages ? a.k_cache[r] : a.q[r], *vc = a.pages ? a.v_cache[r] : a.q[r];
    if (a.pages == 0) continue;
    if (int rc = make_tmap_2d(&p.k[r], kc, mt, 2, D, rows, D, 64, p.box, CU_TENSOR_MAP_SWIZZLE_128B)) return rc;
    if (int rc = make_tmap_2d(&p.v[r], vc, mt, 2, D, rows, D, 64, p.box, CU_TENSOR_MAP_SWIZZLE_128B)) return rc;
  }
  // Tiles are never shared with four units an SM or more: a fifth, unfinished turn costs
  // less than sharing saves.
  const int64_t heads = (int64_t)a.N * a.Hk * p.groups, blocks = a.T / (2 * p.tpt);
  const int64_t sure = (blocks > a.B ? blocks : a.B < a.T ? a.B : a.T) * heads;
  p.few = sure < 4ll * sm_count();
  const int64_t most = (blocks + a.B) * heads;
  const int grid = p.few || most > sm_count() ? sm_count() : (int)most;
  const size_t part = 2 * (D + 2) * kTile * sizeof(float);
  if (int rc = split_workspace(s, p.few ? grid * 2 * part : 0, 2 + (p.few ? grid * 8 : 0), &p.ws, &p.counters))
    return rc;
  auto kern = prefill_kernel<T, D, MAXN>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh<D>::kSmem);
  if (e == cudaSuccess) e = launch_pdl(kern, dim3(grid), dim3(kThreads), Sh<D>::kSmem, s, p);
  if (e != cudaSuccess) return cuda_error(e, "prefill launch");
  note_launch();
  return TP_OK;
}

template <typename T, int D>
int launch_n(const AttnArgs &a, cudaStream_t s) {
  return a.N <= 8 ? launch<T, D, 8>(a, s) : launch<T, D, kMaxShards>(a, s);
}

}  // namespace

int launch_prefill(const AttnArgs &a, cudaStream_t s) {
  if (a.dt == TP_BF16) return a.D == 64 ? launch_n<__nv_bfloat16, 64>(a, s) : launch_n<__nv_bfloat16, 128>(a, s);
  return a.D == 64 ? launch_n<__half, 64>(a, s) : launch_n<__half, 128>(a, s);
}

}  // namespace tp
