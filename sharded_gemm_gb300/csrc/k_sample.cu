// k_sample.cu -- tp_sample: one token per row of logits, from given random
// numbers, with temperature, top-k, top-p and min-p.
//
// With x the row's logits (NaN taken as -inf, +inf as the largest float), M
// their maximum and T the temperature:
//   e_i = exp((x_i - M) * (1/T)),   w_i = floor(e_i * 2^40).
// The weights are whole numbers, so every sum over them is exact and has no
// order: the token does not depend on how the row is split over threads.  What
// a weight below 2^-40 of the largest loses is less than 2^-18 of the total
// for 2^22 tokens.
// The filters keep a prefix of the row sorted by (x descending, index
// ascending): top-k its first k, then top-p those whose weight before them is
// under floor(p * W_k), the first always among them.  The prefix is given by its
// last value and how many of that value (in index order) belong to it, found by
// a radix select on the values' ordered 32-bit keys, with counts for top-k and
// weights for top-p; all elements of one value weigh the same, so a partly kept
// value needs one division.  min-p drops the kept ones with e_i < min_p.
// The token is the first, in index order, whose running weight passes
// floor(u * W).
// Measured: 384 rows of 50272 float32 logits with mixed settings 68 us (floor by
// bytes 11); 152 rows, one an SM: greedy 12, free 15, top-k 50 18, top-k 1000 with
// top-p 25, top-p 36 to 42 us; a single row 9 to 31.
#include "attn.cuh"
#include "ptx.cuh"

#include <atomic>

namespace tp {
namespace {

constexpr int kThreads = 1024;

template <typename T>
__device__ __forceinline__ float logit(const T *p, int64_t i) {
  const float x = static_cast<float>(p[i]);
  return isnan(x) ? -INFINITY : fminf(x, 3.402823466e38f) + 0.0f;  // + 0: one zero
}

// An infinite temperature as the largest finite one: times 0, a -inf would be NaN.
__device__ __forceinline__ float finite(float t) { return t > 3.402823466e38f ? 3.402823466e38f : t; }

// Larger x, larger key.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float ratio(float x, float top, float inv_t) {
  return expf(__fmul_rn(__fsub_rn(x, top), inv_t));
}
__device__ __forceinline__ unsigned long long weight(float e) { return __float2ull_rz(e * 1099511627776.0f); }

// floor(total * share / 2^24), total < 2^62, share <= 2^24
__device__ __forceinline__ unsigned long long part_of(unsigned long long total, unsigned long long share) {
  return (total >> 24) * share + (((total & 0xFFFFFFull) * share) >> 24);
}

// Sum over the block; every thread gets it.
__device__ unsigned long long block_sum(unsigned long long v, unsigned long long *buf) {
#pragma unroll
  for (int m = 16; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  __syncthreads();
  if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = v;
  __syncthreads();
  v = buf[threadIdx.x % 32];
#pragma unroll
  for (int m = 16; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// ---------------------------------------------------------------- rows held on chip
// A row is held as float32 in the shared memory of a cluster of 1, 2, 4 or 8
// CTAs, so the logits are read once.  Thread i of CTA c owns the run of
// elements (c * 1024 + i) * R .. + R - 1, R odd (runs of neighbouring threads
// then start in different banks), and sums over runs in order are sums over the
// row in order.  The end of the last run is padded with -inf.
//
// The end of a kept prefix is narrowed down until a few hundred elements hold it,
// which are put in order on one CTA.
//   top-k: 2048 bins over x count the largest of the threads' runs (of quarters
//     of them for a large k): the bins in which k of those lie hold at least k
//     elements, and not many more.
//   top-p: where it ends is guessed from the row's total as a float and bins that
//     count 4096 of its elements; then one pass sums the exact weights of all and
//     above two values around the guess.  They decide: where the end is not between
//     the two, or too many elements are, weights are summed above seven values
//     between the closest known ones, over the few elements there (a mask of the
//     run's), until it is.  (A miss, about one row in 80, costs 7 us.  Seven fixed
//     values in the first pass and then rounds of seven took 37 to 73 us a wave of
//     152 rows; the guess takes 35 to 42.)
// (Adding every weight to bins in shared memory took 25 us a row: an addition
// costs a lane about two cycles of the SM.)
//
// What bounds it is arithmetic and the joins: of a top-p row's 33 us, 5.5 are the
// load, 3 the float pass, 4 the guess, 7 the exact pass (a logit takes 8 and 35
// instructions), 4 the list, 3 its order, and the rest sums over the block, each a
// barrier or two and 5 to 20 shuffles a warp.

constexpr int kBins = 2048, kList = 2048;
constexpr float kBinScale = 64.0f;  // 1/64 of a logit wide, from the largest down
constexpr int kMarks = 7;  // values above which weights are summed in a round of narrowing
constexpr float kNoWeight = 28.0f;  // so far below the largest a weight is 0
constexpr int kSpread = 1536; // a list this long leaves room for 1024 bins beside it
constexpr int kRanked = 512;  // a list this long is put in order by counting, each element against all
constexpr int kFew = 256;     // and one for which another round of narrowing does not pay
// The end of top-p is guessed from 4096 elements, four of a run.  Counted in those the guess
// is off by up to 15 in the mean square (rows of normal logits, p 0.5 to 0.999); the two
// values around it are kOff away, 1200 elements of 50272 apart.
constexpr int kSamples = 4;
constexpr float kOff = 48.0f;
constexpr int kMaxRun = 51;   // 51 * 1024 floats and RowShared fill a CTA's shared memory; and bits of a mask

typedef unsigned long long u64;

struct alignas(16) RowShared {  // the row's float4 stores begin behind it
  union {
    uint32_t hist[kBins];
    u64 hist64[kBins];
    u64 list[kList];  // filled when the bins have been read
  };
  u64 warp_a[2][32], warp_b[2][32];
  u64 xa[2], xb[2];  // this CTA's sums, exchanged over the cluster
  u64 got[2][3];     // what one thread has read of other CTAs, for all of this one
  uint32_t warp_m[2][32], xm[2];
  uint32_t mark_hi[kMarks + 1][32], mark_lo[kMarks + 1][32];
  u64 mark_sums[kMarks + 1], mark_totals[kMarks + 1];
  u64 answer, before, drawn, bin;
  uint32_t list_n;
};

__device__ __forceinline__ u64 ld_cluster_u64(uint32_t addr) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t atom_cluster_add(uint32_t addr, uint32_t v) {
  uint32_t o;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(o) : "r"(addr), "r"(v) : "memory");
  return o;
}

// floor(e * 2^40), e in [0, 1], summed: the upper and lower 20 bits come out of
// two fused multiply-adds that round toward zero at 2^23, where a float's last
// bit is 1.  The raw bit patterns are added; each carries the pattern of 2^23.
struct WeightSum {
  uint32_t hi = 0, lo = 0;
  int n = 0;
  __device__ __forceinline__ void add(float e) {
    const float t1 = __fmaf_rz(e, 1048576.0f, 8388608.0f);
    const float rest = __fmaf_rn(e, 1048576.0f, -__fsub_rn(t1, 8388608.0f));  // exact
    hi += __float_as_uint(t1);
    lo += __float_as_uint(__fmaf_rz(rest, 1048576.0f, 8388608.0f));
    ++n;
  }
  __device__ __forceinline__ u64 total() const {
    return ((u64)(hi - (uint32_t)n * 0x4B000000u) << 20) + (lo - (uint32_t)n * 0x4B000000u);
  }
};

__device__ __forceinline__ float x_of_key(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
// Orders the row by (x descending, index ascending), without ties.
__device__ __forceinline__ u64 q_of(float x, uint32_t index) { return (u64)order_key(x) << 32 | (uint32_t)~index; }
__device__ __forceinline__ int bin_of(float x, float top) {
  const int b = __float2int_rz((top - x) * kBinScale);
  return b < kBins - 1 ? b : kBins - 1;
}

// A kept prefix: what is above x, and of x itself the indexes up to i.
struct Cut {
  float x;
  uint32_t i;
  __device__ __forceinline__ bool keeps(float v, uint32_t index) const { return v > x || (v == x && index <= i); }
};

// Which elements of a run are meant, one bit each.
struct Mask {
  uint32_t lo = 0, hi = 0;
  __device__ __forceinline__ int count() const { return __popc(lo) + __popc(hi); }
  __device__ __forceinline__ bool any() const { return lo | hi; }
  __device__ __forceinline__ void set(int j, bool on) {
    const uint32_t bit = on ? 1u << (j & 31) : 0;
    if (j < 32) lo |= bit; else hi |= bit;
  }
};
template <typename In>
__device__ __forceinline__ Mask mask_of(int R, In in) {
  Mask m;
  const int n = R < 32 ? R : 32;
#pragma unroll 4
  for (int j = 0; j < n; ++j) m.lo = __funnelshift_r(m.lo, in(j) ? 1u : 0u, 1);
  m.lo = n < 32 ? m.lo >> (32 - n) : m.lo;
#pragma unroll 4
  for (int j = 32; j < R; ++j) m.hi = __funnelshift_r(m.hi, in(j) ? 1u : 0u, 1);
  if (R > 32) m.hi >>= 64 - R;
  return m;
}
// f(j, valid) for the elements of each lane's mask, all lanes of the warp in step:
// a lane that has run out gets j = 0 and valid = false.
template <typename F>
__device__ __forceinline__ void for_each(Mask m, F f) {
  const int most = __reduce_max_sync(0xffffffffu, m.count());
  for (int i = 0; i < most; ++i) {
    const bool low = m.lo != 0;
    const uint32_t w = low ? m.lo : m.hi;
    const int j = w ? (low ? 0 : 32) + __ffs(w) - 1 : 0;
    if (low) m.lo &= m.lo - 1; else m.hi &= m.hi - 1;
    f(j, w != 0);
  }
}

// Weights above N values and of all (the last), as upper and lower 20 bits.
template <int N>
struct MarkSums {
  float mark[N];
  uint32_t hi[N + 1], lo[N + 1];
  __device__ __forceinline__ MarkSums() {
#pragma unroll
    for (int i = 0; i <= N; ++i) hi[i] = lo[i] = 0;
  }
  __device__ __forceinline__ void add(float v, float e) {
    WeightSum w;
    w.add(e);
    const uint32_t h = w.hi - 0x4B000000u, l = w.lo - 0x4B000000u;
    hi[N] += h, lo[N] += l;
#pragma unroll
    for (int i = 0; i < N; ++i)  // the two additions under one predicate
      asm("{\n .reg .pred p;\n setp.gt.f32 p, %2, %3;\n @p add.u32 %0, %0, %4;\n @p add.u32 %1, %1, %5;\n}"
          : "+r"(hi[i]), "+r"(lo[i])
          : "f"(v), "f"(mark[i]), "r"(h), "r"(l));
  }
  __device__ __forceinline__ u64 sum(int i) const { return ((u64)hi[i] << 20) + lo[i]; }
};

struct Row {
  RowShared &sh;
  const float *run;  // this thread's elements
  int R, C, rank;
  uint32_t index0;   // of the run's first element
  float top, inv_t, run_top;
  int par, xpar;  // which of two buffers the next exchange in the block, and over the cluster, uses

  __device__ __forceinline__ void sync() {
    if (C > 1) cluster_sync_all(); else __syncthreads();
  }
  __device__ __forceinline__ uint32_t at0(const void *p) { return mapa_shared(smem_u32(p), 0); }
  // Where the draw goes, for resolve().
  u64 share;
  float min_p, logz;
  int64_t *token;
  float *logprob;
  bool drawn;
  // What rank 0 left in a and b before a sync, in every thread.
  __device__ __forceinline__ void from_rank0(const u64 &at_a, const u64 &at_b, u64 &a, u64 &b) {
    if (C > 1) {
      if (threadIdx.x == 0) sh.got[xpar][0] = ld_cluster_u64(at0(&at_a)), sh.got[xpar][1] = ld_cluster_u64(at0(&at_b));
      __syncthreads();
      a = sh.got[xpar][0], b = sh.got[xpar][1];
      xpar ^= 1;
    } else {
      a = at_a, b = at_b;
    }
  }
  __device__ __forceinline__ float e_of(float x) { return ratio(x, top, inv_t); }

  // Sums of a and b over the cluster; every thread gets them, and in before_a
  // the sum of the CTAs of lower rank.
  __device__ __forceinline__ void reduce(u64 &a, u64 &b, u64 *before_a = nullptr) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int m = 16; m > 0; m /= 2) {
      a += __shfl_xor_sync(0xffffffffu, a, m);
      b += __shfl_xor_sync(0xffffffffu, b, m);
    }
    if (lane == 0) sh.warp_a[par][warp] = a, sh.warp_b[par][warp] = b;
    __syncthreads();
    a = sh.warp_a[par][lane], b = sh.warp_b[par][lane];
#pragma unroll
    for (int m = 16; m > 0; m /= 2) {
      a += __shfl_xor_sync(0xffffffffu, a, m);
      b += __shfl_xor_sync(0xffffffffu, b, m);
    }
    if (before_a) *before_a = 0;
    if (C > 1) {
      if (threadIdx.x == 0) sh.xa[xpar] = a, sh.xb[xpar] = b;
      cluster_sync_all();
      // one warp reads the other CTAs' (all threads reading took 2 us at 8 CTAs)
      if (warp == 0) {
        a = lane < C ? ld_cluster_u64(mapa_shared(smem_u32(&sh.xa[xpar]), lane)) : 0;
        b = lane < C ? ld_cluster_u64(mapa_shared(smem_u32(&sh.xb[xpar]), lane)) : 0;
        u64 lower = lane < rank ? a : 0;
#pragma unroll
        for (int m = 4; m > 0; m /= 2) {
          a += __shfl_xor_sync(0xffffffffu, a, m);
          b += __shfl_xor_sync(0xffffffffu, b, m);
          lower += __shfl_xor_sync(0xffffffffu, lower, m);
        }
        if (lane == 0) sh.got[xpar][0] = a, sh.got[xpar][1] = b, sh.got[xpar][2] = lower;
      }
      __syncthreads();
      a = sh.got[xpar][0], b = sh.got[xpar][1];
      if (before_a) *before_a = sh.got[xpar][2];
      xpar ^= 1;
    }
    par ^= 1;
  }
  // The largest (or with ADD the sum) of v over the cluster.
  template <bool ADD>
  static __device__ __forceinline__ uint32_t of_warp(uint32_t v) {
    return ADD ? __reduce_add_sync(0xffffffffu, v) : __reduce_max_sync(0xffffffffu, v);
  }
  template <bool ADD>
  __device__ __forceinline__ uint32_t reduce_u32(uint32_t v) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    v = of_warp<ADD>(v);
    if (lane == 0) sh.warp_m[par][warp] = v;
    __syncthreads();
    v = of_warp<ADD>(sh.warp_m[par][lane]);
    if (C > 1) {
      if (threadIdx.x == 0) sh.xm[xpar] = v;
      cluster_sync_all();
      if (warp == 0) {
        v = of_warp<ADD>(lane < C ? ld_cluster_u32(mapa_shared(smem_u32(&sh.xm[xpar]), lane)) : 0);
        if (lane == 0) sh.got[xpar][0] = v;
      }
      __syncthreads();
      v = (uint32_t)sh.got[xpar][0];
      xpar ^= 1;
    }
    par ^= 1;
    return v;
  }
  __device__ __forceinline__ uint32_t reduce_max(uint32_t v) { return reduce_u32<false>(v); }
  __device__ __forceinline__ uint32_t reduce_count(uint32_t v) { return reduce_u32<true>(v); }
  // Sum over the block of the values of lower threads.
  __device__ __forceinline__ u64 scan_before(u64 v, u64 &total) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    u64 run = v;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
      const u64 o = __shfl_up_sync(0xffffffffu, run, m);
      if (lane >= m) run += o;
    }
    if (lane == 31) sh.warp_a[par][warp] = run;
    __syncthreads();
    const u64 w = sh.warp_a[par][lane];
    u64 base = lane < warp ? w : 0;
    total = w;
#pragma unroll
    for (int m = 16; m > 0; m /= 2) {
      base += __shfl_xor_sync(0xffffffffu, base, m);
      total += __shfl_xor_sync(0xffffffffu, total, m);
    }
    par ^= 1;
    return base + run - v;
  }

  // The threads' mark sums over the cluster; every thread gets them.  A thread's
  // halves are below 2^26 (64 elements of 2^20), a warp's below 2^31.
  template <int N>
  __device__ __forceinline__ void reduce_marks(const MarkSums<N> &m, u64 (&v)[N + 1]) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int i = 0; i <= N; ++i) {
      const uint32_t h = __reduce_add_sync(0xffffffffu, m.hi[i]), l = __reduce_add_sync(0xffffffffu, m.lo[i]);
      if (lane == 0) sh.mark_hi[i][warp] = h, sh.mark_lo[i][warp] = l;
    }
    __syncthreads();
    if (warp <= N) {
      u64 x = ((u64)sh.mark_hi[warp][lane] << 20) + sh.mark_lo[warp][lane];
#pragma unroll
      for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane == 0) (C > 1 ? sh.mark_sums : sh.mark_totals)[warp] = x;
    }
    sync();
    if (C > 1) {
      if (warp <= N) {
        u64 x = lane < C ? ld_cluster_u64(mapa_shared(smem_u32(&sh.mark_sums[warp]), lane)) : 0;
#pragma unroll
        for (int o = 4; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0) sh.mark_totals[warp] = x;
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i <= N; ++i) v[i] = sh.mark_totals[i];
  }

  // Before bins are added to: the last readers of what they share memory with
  // are a sync behind.
  __device__ __forceinline__ void clear_bins() {
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.hist64[i] = 0;
    if (threadIdx.x == 0) sh.list_n = 0, sh.bin = kBins - 1, sh.before = 0;
    __syncthreads();
  }
  // The bin over the cluster in which the running total reaches `target`, and the total before it.
  template <typename H>
  __device__ __forceinline__ int pick_bin(const H *hist, u64 target, u64 &below) {
    sync();  // every CTA's bins are complete
    const int per = C == 1 ? 2 : 1, i = rank * (kBins / C) + (int)threadIdx.x * per;
    u64 h0 = 0, h1 = 0;
    if ((int)threadIdx.x * per < kBins / C) {
      if (C == 1) {
        h0 = hist[i], h1 = hist[i + 1];
      } else {
        for (int c = 0; c < C; ++c) {
          const uint32_t at = mapa_shared(smem_u32(hist + i), c);
          h0 += sizeof(H) == 4 ? ld_cluster_u32(at) : ld_cluster_u64(at);
        }
      }
    }
    u64 all, before = scan_before(h0 + h1, all), base = 0, unused = 0;
    if (C > 1) {
      u64 mine = threadIdx.x == 0 ? all : 0;
      reduce(mine, unused, &base);
    }
    const u64 c0 = base + before, c1 = c0 + h0, c2 = c1 + h1;
    auto mark = [&](u64 from, u64 to, int at) {
      if (from < target && to >= target) {
        st_cluster_u64(at0(&sh.bin), at);
        st_cluster_u64(at0(&sh.before), from);
      }
    };
    mark(c0, c1, i);
    mark(c1, c2, i + 1);
    sync();
    u64 bin;
    from_rank0(sh.before, sh.bin, below, bin);
    return (int)bin;
  }

  // Puts this thread's elements of `mask` on rank 0's list (cleared a sync before).
  __device__ __forceinline__ void gather(const Mask &mask) {
    if (__any_sync(0xffffffffu, mask.any())) {
      // the warp's places, then the lane's among them
      const int lane = threadIdx.x % 32;
      const uint32_t mine = mask.count();
      uint32_t at = mine;
#pragma unroll
      for (int m = 1; m < 32; m *= 2) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, at, m);
        if (lane >= m) at += o;
      }
      uint32_t base = 0;
      if (lane == 31) base = C > 1 ? atom_cluster_add(at0(&sh.list_n), at) : atomicAdd(&sh.list_n, at);
      at += __shfl_sync(0xffffffffu, base, 31) - mine;
      for_each(mask, [&](int j, bool valid) {
        if (valid) st_cluster_u64(at0(&sh.list[at++]), q_of(run[j], index0 + j));
      });
    }
    sync();
  }
  __device__ __forceinline__ void clear_list() {
    if (threadIdx.x == 0) sh.list_n = 0;
    sync();
  }

  // Puts rank 0's list in order, the largest first.  No element is above `from`,
  // and none further below it than `reach` (infinity: not known).
  __device__ __forceinline__ void order_list(int n, float from, float reach) {
    const int tid = threadIdx.x;
    if (n <= kRanked) {
      const u64 q = tid < n ? sh.list[tid] : 0;
      int place = 0;
      if (tid < n) {
#pragma unroll 4
        for (int j = 0; j < n; ++j) place += sh.list[j] > q;
      }
      __syncthreads();
      if (tid < n) sh.list[place] = q;
      __syncthreads();
      return;
    }
    if (n <= kSpread && reach < INFINITY) {
      // 1024 bins over the reach, elements to their bins, then each among its bin's few
      uint32_t *bins = reinterpret_cast<uint32_t *>(sh.list + kSpread);
      const float scale = kThreads / reach;
      auto bin = [&](u64 q) {
        const int b = __float2int_rz((from - x_of_key((uint32_t)(q >> 32))) * scale);
        return b < kThreads - 1 ? b : kThreads - 1;
      };
      bins[tid] = 0;
      __syncthreads();
      u64 q[2];
      int b[2], place[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        q[i] = tid + i * kThreads < n ? sh.list[tid + i * kThreads] : 0;
        b[i] = bin(q[i]);
        place[i] = 0;
        if (q[i]) place[i] = atomicAdd(&bins[b[i]], 1u);
      }
      __syncthreads();
      u64 all;
      const uint32_t mine = bins[tid], before = (uint32_t)scan_before(mine, all);
      par ^= 1;  // as on the other CTAs
      __syncthreads();
      bins[tid] = before << 16 | (before + mine);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (q[i]) sh.list[(bins[b[i]] >> 16) + place[i]] = q[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int lo = bins[b[i]] >> 16, hi = bins[b[i]] & 0xffff;
        place[i] = lo;
        if (q[i])
          for (int j = lo; j < hi; ++j) place[i] += sh.list[j] > q[i];
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (q[i]) sh.list[place[i]] = q[i];
      __syncthreads();
      return;
    }
    int size = 2;
    while (size < n) size *= 2;
    for (int i = n + tid; i < size; i += kThreads) sh.list[i] = 0;
    __syncthreads();
    for (int width = 2; width <= size; width *= 2)
      for (int step = width / 2; step > 0; step /= 2) {
        if (tid < size / 2) {
          const int i = (tid & ~(step - 1)) << 1 | (tid & (step - 1));
          const u64 x = sh.list[i], y = sh.list[i + step];
          if ((x < y) == ((i & width) == 0)) sh.list[i] = y, sh.list[i + step] = x;
        }
        __syncthreads();
      }
  }

  // Rank 0's list: n elements, all of a stretch of the order behind which
  // `place0` elements of weight `above` lie.  The cut that keeps the first k of
  // the order and, by_p, of those the ones whose weight before them is under
  // `want`.  A list that begins the order (whole): want is part_of(the k's
  // weight, p_share), and where all that is kept is on the list, few enough, the
  // token is drawn from it at once (drawn).
  __device__ __forceinline__ Cut resolve(int n, u64 place0, u64 above, u64 k, bool by_p, u64 want, float from,
                                         float reach, bool whole = false, u64 p_share = 0) {
    if (rank == 0) {
      const int tid = threadIdx.x;
      __syncthreads();
      order_list(n, from, reach);
      u64 q[2], w[2];
      float e[2];
      bool in[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = 2 * tid + i;
        in[i] = at < n && place0 + at < k;
        q[i] = at < n ? sh.list[at] : 0;
        e[i] = in[i] ? e_of(x_of_key((uint32_t)(q[i] >> 32))) : 0.0f;
        w[i] = weight(e[i]);
      }
      u64 total;
      const u64 before = above + scan_before(w[0] + w[1], total);
      par ^= 1;  // as on the other CTAs
      if (by_p) {
        if (whole) want = part_of(total, p_share);
        in[0] = in[0] && (before < want || place0 + 2 * tid == 0);
        in[1] = in[1] && before + w[0] < want;
      }
      const int kept = __syncthreads_count(in[0]) + __syncthreads_count(in[1]);
      if (tid == 0) sh.answer = sh.list[kept - 1], sh.drawn = 0;
      if (whole && n <= kList / 2 && kept <= kRanked) {
        // the draw: the kept ones' weights beside them, then each sums those of lower index
        u64 *kept_w = sh.list + kList / 2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (e[i] < min_p) w[i] = 0;
          if (!in[i]) w[i] = 0;
          if (2 * tid + i < kept) kept_w[2 * tid + i] = w[i];
        }
        u64 sum;
        scan_before(w[0] + w[1], sum);
        par ^= 1;
        __syncthreads();
        const u64 r = part_of(sum, share);
        if (tid < kept) {
          const u64 mine = sh.list[tid];
          const uint32_t index = ~(uint32_t)mine;
          u64 run = 0;
#pragma unroll 4
          for (int j = 0; j < kept; ++j) run += ~(uint32_t)sh.list[j] < index ? kept_w[j] : 0;
          if (run <= r && r < run + kept_w[tid]) {
            *token = index;
            if (logprob) *logprob = x_of_key((uint32_t)(mine >> 32)) - top - logz;
          }
        }
        if (tid == 0) sh.drawn = 1;
      }
    }
    sync();
    u64 q, was_drawn;
    from_rank0(sh.answer, sh.drawn, q, was_drawn);
    drawn = was_drawn != 0;
    return Cut{x_of_key((uint32_t)(q >> 32)), ~(uint32_t)q};
  }

  // The cut behind which the stretch [lo, hi] of the order ends the prefix:
  // rounds of 2048 equal parts of the stretch.  For rows of many equal or
  // near-equal values.
  template <bool BY_WEIGHT>
  __device__ __noinline__ Cut select_in(u64 lo, u64 hi, u64 above, u64 want) {
    for (;;) {
      const int bits = 64 - __clzll((hi - lo) | 1), shift = bits > 11 ? bits - 11 : 0;
      clear_bins();
      for (int j = 0; j < R; ++j) {
        const u64 q = q_of(run[j], index0 + j);
        if (q < lo || q > hi) continue;
        const u64 add = BY_WEIGHT ? weight(e_of(run[j])) : 1;
        if (add) atomicAdd(&sh.hist64[(hi - q) >> shift], add);
      }
      u64 below;
      const int picked = pick_bin(sh.hist64, want - above, below);
      above += below;
      const u64 new_hi = hi - ((u64)picked << shift), span = (1ull << shift) - 1;
      const u64 new_lo = new_hi - lo > span ? new_hi - span : lo;
      lo = new_lo, hi = new_hi;
      const Mask mask = mask_of(R, [&](int j) {
        const u64 q = q_of(run[j], index0 + j);
        return q >= lo && q <= hi;
      });
      const uint32_t n = reduce_count(mask.count());
      if (n <= kList) {
        gather(mask);
        return BY_WEIGHT ? resolve((int)n, 1, above, ~0ull, true, want, top, INFINITY)
                         : resolve((int)n, above, 0, want, false, 0, top, INFINITY);
      }
    }
  }

  // The first k, and of those with by_p the ones under part_of(their weight, p_share).
  __device__ __forceinline__ Cut select_count(u64 k, bool by_p, u64 p_share, bool &only_first) {
    // k runs (or quarters) whose largest is in one of the first bins hold k elements in them
    int limit = kBins - 1;
    u64 below = 0;
    auto in_bins = [&](float v) { return limit == kBins - 1 || (top - v) * kBinScale < (float)(limit + 1); };
    const int parts = k <= (u64)C * kThreads / 4 ? 1 : 4;
    if (k <= (u64)C * kThreads * parts) {
      clear_bins();
      if (parts == 1) {
        atomicAdd(&sh.hist[bin_of(run_top, top)], 1u);
      } else {
        for (int i = 0; i < 4; ++i) {
          float most = -INFINITY;
          for (int j = R * i / 4; j < R * (i + 1) / 4; ++j) most = fmaxf(most, run[j]);
          if (most > -INFINITY) atomicAdd(&sh.hist[bin_of(most, top)], 1u);
        }
      }
      limit = pick_bin(sh.hist, k, below);
    }
    Mask mask;
    if (in_bins(run_top)) mask = mask_of(R, [&](int j) { return in_bins(run[j]); });
    u64 n = reduce_count(mask.count()), over = 0;
    if (n > kList) {
      clear_bins();
      for_each(mask, [&](int j, bool valid) {
        if (valid) atomicAdd(&sh.hist[bin_of(run[j], top)], 1u);
      });
      limit = pick_bin(sh.hist, k, over);
      Mask equal, under;
      for_each(mask, [&](int j, bool valid) {
        const int b = bin_of(run[j], top);
        equal.set(j, valid && b == limit);
        under.set(j, valid && b < limit);
      });
      n = reduce_count(equal.count());
      mask = equal;
      if (n + over <= kList) {
        n += over, over = 0;
        mask.lo |= under.lo, mask.hi |= under.hi;
      }
    }
    Cut cut;
    if (n <= kList) {
      clear_list();
      gather(mask);
      const bool whole = over == 0;
      const float reach = whole && limit < kBins - 1 ? (limit + 1) / kBinScale : INFINITY;
      cut = resolve((int)n, over, 0, k, by_p && whole, 0, top, reach, whole, p_share);
      if (drawn || (by_p && whole)) return cut;
    } else {
      u64 lo, hi;
      stretch(limit, lo, hi);
      cut = select_in<false>(lo, hi, over, k);
    }
    u64 run_above = 0;
    return by_p ? select_weight(0, p_share, cut, top, -INFINITY, 0, false, only_first, run_above, mask) : cut;
  }

  // The stretch of the order that the elements of a bin take.
  __device__ __forceinline__ void stretch(int bin, u64 &lo, u64 &hi) {
    uint32_t most = 0, not_least = 0;
    for (int j = 0; j < R; ++j) {
      const uint32_t key = order_key(run[j]);
      if (bin_of(run[j], top) != bin) continue;
      if (key > most) most = key;
      if (~key > not_least) not_least = ~key;
    }
    hi = (u64)reduce_max(most) << 32 | 0xffffffffu;
    lo = (u64)~reduce_max(not_least) << 32;
  }

  // Counts the samples, kSamples elements of every C-th thread's run, in rank 0's
  // bins (cleared a sync before) over the values that have a weight.
  __device__ __forceinline__ void sample() {
    if (threadIdx.x % C) return;
    const float scale = inv_t * (kBins / kNoWeight);
    const int n = min(R, kSamples), step = R / n;
    for (int i = 0; i < n; ++i) {
      const int b = min(__float2int_rz((top - run[i * step]) * scale), kBins - 1);
      if (C > 1) atom_cluster_add(at0(&sh.hist[b]), 1u); else atomicAdd(&sh.hist[b], 1u);
    }
  }
  // Guesses where the weight below falls to `rest` of a row, by the samples (counted a
  // sync before): values a little above and below.  All samples of a bin are taken
  // to weigh what its middle does.
  __device__ __forceinline__ void guess(u64 rest, float &high, float &low) {
    if (rank == 0) {
      const int tid = threadIdx.x;
      const float width = fminf(__fdiv_rn(kNoWeight / kBins, inv_t), 1e30f);  // times 0 a number
      const uint32_t n0 = sh.hist[2 * tid], n1 = sh.hist[2 * tid + 1];
      auto mass = [&](int i, uint32_t n) {
        const float e = exp2f((i + 0.5f) * (-kNoWeight / kBins * 1.4426950408889634f));
        return i == kBins - 1 ? 0 : (u64)((float)n * e * 68719476736.0f);
      };
      const u64 m0 = mass(2 * tid, n0), m1 = mass(2 * tid + 1, n1);
      // weights (below 2^48, in units of 2^-36) and counts (up to 4096) in one number
      u64 both;
      const u64 both_before = scan_before((m0 + m1) << 13 | (n0 + n1), both);
      par ^= 1;  // as on the other CTAs
      const u64 m_before = both_before >> 13, total = both >> 13;
      const uint32_t before = both_before & 8191, samples = both & 8191;
      rest = (rest >> 4) / (uint32_t)R * min(R, kSamples) / C;
      const u64 target = total > rest ? total - rest : 0;
      if (tid == 0) sh.answer = __float_as_uint((float)samples);
      __syncthreads();
      auto at = [&](u64 m_from, u64 m, float n_from, uint32_t n) {
        if (target >= m_from && target - m_from < m)
          sh.answer = __float_as_uint(n_from + (float)n * ((float)(target - m_from) / (float)m));
      };
      at(m_before, m0, before, n0);
      at(m_before + m0, m1, before + n0, n1);
      if (tid == 0) sh.before = __float_as_uint(top), sh.bin = __float_as_uint(top - kBins * width);
      __syncthreads();
      const float place = __uint_as_float((uint32_t)sh.answer);
      auto mark = [&](float rank_at, u64 &to, int i, float n_from, uint32_t n) {
        if (n && rank_at >= n_from && rank_at < n_from + n)
          to = __float_as_uint(top - ((float)i + (rank_at - n_from) / (float)n) * width);
      };
      mark(place - kOff, sh.before, 2 * tid, before, n0);
      mark(place - kOff, sh.before, 2 * tid + 1, before + n0, n1);
      mark(place + kOff, sh.bin, 2 * tid, before, n0);
      mark(place + kOff, sh.bin, 2 * tid + 1, before + n0, n1);
    }
    sync();
    u64 h, l;
    from_rank0(sh.before, sh.bin, h, l);
    high = __uint_as_float((uint32_t)h), low = __uint_as_float((uint32_t)l);
  }

  // Of what `from` keeps (weight `total`, 0: not known) the ones whose weight
  // before them is under part_of(total, p_share).  The end is known to lie among
  // the values in (low, high], with weight `above` over them, run_above of it
  // this thread's, and this thread's elements there in `mask` if `masked`.  On
  // return `mask` has its elements of the last such stretch, and run_above fits it.
  __device__ __noinline__ Cut select_weight(u64 total, u64 p_share, Cut from, float high, float low, u64 above,
                                            bool masked, bool &only_first, u64 &run_above, Mask &mask) {
    if (total == 0) {
      u64 unused = 0;
      WeightSum sum;
      for (int j = 0; j < R; ++j) sum.add(from.keeps(run[j], index0 + j) ? e_of(run[j]) : 0.0f);
      total = sum.total();
      reduce(total, unused);
    }
    const u64 want = part_of(total, p_share);
    if (want == 0) {
      only_first = true;
      return from;
    }
    if (masked) {
    } else if (from.x == -INFINITY) mask = mask_of(R, [&](int j) { return run[j] <= high && run[j] > low; });
    else mask = mask_of(R, [&](int j) { return run[j] <= high && run[j] > low && from.keeps(run[j], index0 + j); });
    const float floor_x = __fdiv_rn(-kNoWeight, inv_t) + top;
    uint32_t n = reduce_count(mask.count()), was = ~0u;
    while (n > (low > -INFINITY ? kSpread : kFew) && n < was) {
      // the weights above kMarks values between low and high
      const float from_x = low > floor_x ? low : floor_x, step = (high - from_x) * (1.0f / (kMarks + 1));
      MarkSums<kMarks> m;
#pragma unroll
      for (int i = 0; i < kMarks; ++i) m.mark[i] = high - (i + 1) * step;
      for_each(mask, [&](int j, bool valid) {
        const float x = run[j];
        m.add(x, valid ? e_of(x) : 0.0f);
      });
      u64 v[kMarks + 1], over = 0, run_over = 0;
      reduce_marks(m, v);
#pragma unroll
      for (int i = 0; i < kMarks; ++i) {
        if (above + v[i] < want) high = m.mark[i], over = v[i], run_over = m.sum(i);
        if (above + v[kMarks - 1 - i] >= want) low = m.mark[kMarks - 1 - i];
      }
      above += over, run_above += run_over;
      Mask kept;
      for_each(mask, [&](int j, bool valid) { kept.set(j, valid && run[j] <= high && run[j] > low); });
      mask = kept;
      was = n;
      n = reduce_count(mask.count());
    }
    if (n <= kList) {
      clear_list();
      gather(mask);
      return resolve((int)n, above ? 1 : 0, above, ~0ull, true, want, high, high - low);
    }
    u64 lo = ((u64)order_key(low) + 1) << 32;
    const u64 from_q = q_of(from.x, from.i);
    if (lo < from_q) lo = from_q;
    return select_in<true>(lo, (u64)order_key(high) << 32 | 0xffffffffu, above, want);
  }
};

// The row that cluster `b` takes: the rows whose filters take several passes
// come first, so that a batch of more rows than the GPU holds at once does not
// end on them (384 mixed rows of 50272: 126 us in the order given).
__device__ __forceinline__ int64_t row_of(const SampleArgs &a, RowShared &sh, int64_t b) {
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  auto slow = [&](int64_t row) {
    const float t = a.temperature ? a.temperature[row] : 1.0f, p = a.top_p ? a.top_p[row] : 1.0f;
    const int k = a.top_k ? a.top_k[row] : 0;
    return t >= 9.5367431640625e-7f && (k <= 0 || k > a.V ? p < 1.0f : k > kFew);
  };
  int64_t slow_rows = 0;
  for (int64_t base = 0; base < a.B; base += kThreads)
    slow_rows += __syncthreads_count(base + tid < a.B && slow(base + tid));
  const bool of_slow = b < slow_rows;
  int64_t target = of_slow ? b : b - slow_rows;  // the row's place among its kind
  for (int64_t base = 0; base < a.B; base += kThreads) {
    const bool mine = base + tid < a.B && slow(base + tid) == of_slow;
    const uint32_t ballot = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) sh.warp_m[0][warp] = __popc(ballot);
    __syncthreads();
    const uint32_t n = sh.warp_m[0][lane];
    const int before = (int)__reduce_add_sync(0xffffffffu, lane < warp ? n : 0) + __popc(ballot & ((1u << lane) - 1));
    if (mine && before == target) sh.answer = base + tid;
    target -= (int)__reduce_add_sync(0xffffffffu, n);
    __syncthreads();
  }
  return (int64_t)sh.answer;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    sample_row_kernel(const __grid_constant__ SampleArgs a, int C, int R, bool reorder) {
  extern __shared__ __align__(16) uint8_t smem[];
  RowShared &sh = *reinterpret_cast<RowShared *>(smem);
  float *xs = reinterpret_cast<float *>(smem + sizeof(RowShared));
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t b = reorder ? row_of(a, sh, blockIdx.x / C) : blockIdx.x / C;
  const int rank = blockIdx.x % C, slice = R * kThreads;
  const T *x = static_cast<const T *>(a.logits) + b * a.ld + (int64_t)rank * slice;
  const int64_t left = a.V - (int64_t)rank * slice;
  const int n = left < 0 ? 0 : left < slice ? (int)left : slice;

  const float t = a.temperature ? finite(a.temperature[b]) : 1.0f, u = a.u[b];
  const bool greedy = !(t >= 9.5367431640625e-7f);
  long long k = greedy ? 1 : (a.top_k ? a.top_k[b] : 0);
  if (k <= 0 || k > a.V) k = a.V;
  const float p = a.top_p ? a.top_p[b] : 1.0f;
  const bool by_p = p < 1.0f;
  const u64 p_share = (u64)(fmaxf(p, 0.0f) * 16777216.0f);
  float min_p = a.min_p ? a.min_p[b] : 0.0f;
  min_p = min_p > 0.0f ? fminf(min_p, 1.0f) : 0.0f;

  // ---- the slice into shared memory, and its largest
  float top = -INFINITY;
  auto clean = [](float v) { return isnan(v) ? -INFINITY : fminf(v, 3.402823466e38f) + 0.0f; };
  constexpr int kVec = 16 / sizeof(T);
  const int vecs = (uintptr_t)x % 16 == 0 ? n / kVec : 0;
#pragma unroll 4
  for (int i = tid; i < vecs; i += kThreads) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(x) + i);
    const uint32_t bits[4] = {v.x, v.y, v.z, v.w};
    float f[kVec];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 4) {
        f[j] = clean(__uint_as_float(bits[j]));
      } else {
        const float2 pair = Half2<T>::unpack(bits[j]);
        f[2 * j] = clean(pair.x), f[2 * j + 1] = clean(pair.y);
      }
    }
#pragma unroll
    for (int j = 0; j < kVec; j += 4) {
      *reinterpret_cast<float4 *>(xs + i * kVec + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
      top = fmaxf(top, fmaxf(fmaxf(f[j], f[j + 1]), fmaxf(f[j + 2], f[j + 3])));
    }
  }
  for (int i = vecs * kVec + tid; i < slice; i += kThreads) {
    const float v = i < n ? clean(static_cast<float>(x[i])) : -INFINITY;
    xs[i] = v;
    top = fmaxf(top, v);
  }
  const bool by_k = k < a.V || k == 1, free_draw = !by_k && !by_p, guessed = !by_k && by_p && p_share > 0;
  Row row{sh, xs + tid * R, R, C, rank, (uint32_t)(rank * slice + tid * R), 0.0f, greedy ? 1.0f : 1.0f / t, -INFINITY, 0,
          0};
  row.drawn = false;
  if (guessed) row.clear_bins();
  row.top = top = x_of_key(row.reduce_max(order_key(top)));  // also: the slice is in shared memory
  if (top == -INFINITY) {  // nothing can be drawn
    if (rank == 0 && tid == 0) {
      a.tokens[b] = -1;
      if (a.logprobs) a.logprobs[b] = -INFINITY;
    }
    if (C > 1) cluster_sync_all();
    return;
  }

  // ---- the row's own softmax total z, and in the same pass the exact weights it is drawn by,
  // or with top-p alone their total zt as a float and samples
  float z = 0.0f, zt = 0.0f;
  WeightSum sum;  // what is kept of the run, where that is known
  // (where the temperature is 1, z's terms are the weights' own)
  const bool own = row.inv_t == 1.0f;
  auto exp2_of = [](float v) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
  };
  auto z_of = [&](float v) { return exp2_of((v - top) * 1.4426950408889634f); };
  if (free_draw) {
#pragma unroll 4
    for (int j = 0; j < R; ++j) {
      const float v = row.run[j], e = row.e_of(v);
      z += own ? e : z_of(v);
      sum.add(e < min_p ? 0.0f : e);
    }
  } else if (guessed && !own) {
    row.sample();
    const float scale = row.inv_t * 1.4426950408889634f;
#pragma unroll 4
    for (int j = 0; j < R; ++j) {
      const float v = row.run[j];
      z += z_of(v);
      zt += exp2_of((v - top) * scale);
      row.run_top = fmaxf(row.run_top, v);
    }
  } else {
    if (guessed) row.sample();
#pragma unroll 4
    for (int j = 0; j < R; ++j) {
      const float v = row.run[j];
      z += z_of(v);
      row.run_top = fmaxf(row.run_top, v);
    }
  }
  // the threads' sums are joined as whole numbers of 2^-40, which have no order
  u64 zsum = (u64)(z * 1099511627776.0f), ztsum = (u64)(zt * 1099511627776.0f), unused;
  row.reduce(zsum, ztsum);
  if (own) ztsum = zsum;
  const float logz = logf((float)zsum * 9.094947017729282e-13f);
  row.share = u > 0.0f ? (u64)(fminf(u, 1.0f) * 16777216.0f) : 0ull;
  if (row.share > 16777215ull) row.share = 16777215ull;
  row.min_p = min_p, row.logz = logz, row.token = a.tokens + b, row.logprob = a.logprobs ? a.logprobs + b : nullptr;

  // ---- the kept prefix
  Cut cut{-INFINITY, 0xffffffffu};
  bool only_first = k == 1 || (by_p && p_share == 0);
  u64 mine = sum.total();
  bool summed = free_draw;
  if (!only_first && by_k) {
    cut = row.select_count((u64)k, by_p, p_share, only_first);
    if (row.drawn) {
      if (C > 1) cluster_sync_all();
      return;
    }
  } else if (!only_first && by_p) {
    float high, low;
    row.guess((u64)((1.0f - p) * (float)ztsum), high, low);
    // the exact weights of all, and of what is above the two values; which lie between
    MarkSums<2> marks;
    marks.mark[0] = high, marks.mark[1] = low;
    Mask mask = mask_of(R, [&](int j) {
      const float v = row.run[j];
      marks.add(v, row.e_of(v));
      return v <= high && v > low;
    });
    u64 v[3], above = 0, run_above = 0;
    row.reduce_marks(marks, v);
    const u64 want = part_of(v[2], p_share);
    const bool hit = v[0] < want && v[1] >= want;
    if (hit) above = v[0], run_above = marks.sum(0);
    else if (v[0] >= want) low = high, high = top;
    else high = low, low = -INFINITY, above = v[1], run_above = marks.sum(1);
    cut = row.select_weight(v[2], p_share, cut, high, low, above, hit, only_first, run_above, mask);
    if (!(min_p > 0.0f)) {  // all above the last stretch is kept, and of it what the cut keeps
      summed = true;
      mine = run_above;
      for_each(mask, [&](int j, bool valid) {
        const float x = row.run[j];
        mine += valid && cut.keeps(x, row.index0 + j) ? weight(row.e_of(x)) : 0;
      });
    }
  }
  if (only_first) {
    uint32_t best = 0;
    if (row.run_top == top) {
      int j = 0;
      while (row.run[j] != top) ++j;
      best = ~(row.index0 + j);
    }
    best = row.reduce_max(best);
    if (rank == 0 && tid == 0) {
      a.tokens[b] = ~best;
      if (a.logprobs) a.logprobs[b] = -logz;
    }
    if (C > 1) cluster_sync_all();
    return;
  }

  // ---- the draw
  auto kept_e = [&](int j) {
    const float v = row.run[j], e = row.e_of(v);
    return cut.keeps(v, row.index0 + j) && !(e < min_p) ? e : 0.0f;
  };
  if (!summed) {
    // what may be kept: from the cut up, and nothing clearly below min_p's value (its
    // logarithm, with a margin above the error of the exponential and of this line)
    float from = cut.x;
    if (min_p > 0.0f) from = fmaxf(from, top + (logf(min_p) - 1e-3f) * t - 1e-5f * fabsf(top));
    sum = WeightSum();
    for_each(mask_of(R, [&](int j) { return row.run[j] >= from; }),
             [&](int j, bool valid) { sum.add(valid ? kept_e(j) : 0.0f); });
    mine = sum.total();
  }
  u64 block, total, before = row.scan_before(mine, block), lower;
  total = tid == 0 ? block : 0;
  unused = 0;
  if (C > 1) {
    row.reduce(total, unused, &lower);
    before += lower;
  } else {
    total = block;
  }
  const u64 r = part_of(total, row.share);
  const uint32_t hit = __ballot_sync(0xffffffffu, r >= before && r < before + mine);
  if (hit) {
    // this warp holds the run: its elements 32 at a time
    const int l = __ffs(hit) - 1;
    row.run = xs + (warp * 32 + l) * R;
    row.index0 = rank * slice + (warp * 32 + l) * R;
    u64 at = __shfl_sync(0xffffffffu, before, l);
    for (int j0 = 0; j0 < R; j0 += 32) {
      const int j = j0 + lane;
      u64 w = j < R ? weight(kept_e(j)) : 0;
#pragma unroll
      for (int m = 1; m < 32; m *= 2) {
        const u64 o = __shfl_up_sync(0xffffffffu, w, m);
        if (lane >= m) w += o;
      }
      const uint32_t found = __ballot_sync(0xffffffffu, at + w > r);
      if (found) {
        if (lane == __ffs(found) - 1) {
          a.tokens[b] = row.index0 + j;
          if (a.logprobs) a.logprobs[b] = row.run[j] - top - logz;
        }
        break;
      }
      at += __shfl_sync(0xffffffffu, w, 31);
    }
  }
  if (C > 1) cluster_sync_all();  // no CTA leaves while another may still read its shared memory
}

// ---------------------------------------------------------------- longer rows
template <typename T>
__global__ void __launch_bounds__(kThreads) sample_wide_kernel(const __grid_constant__ SampleArgs a) {
  __shared__ unsigned long long buf[32], hist[256];
  __shared__ float fbuf[32];
  __shared__ unsigned long long pick_before;
  __shared__ uint32_t pick_digit;
  griddep_wait();
  const int64_t b = blockIdx.x;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const T *x = static_cast<const T *>(a.logits) + b * a.ld;
  const int64_t V = a.V;

  float top = -INFINITY;
  for (int64_t i = tid; i < V; i += kThreads) top = fmaxf(top, logit(x, i));
#pragma unroll
  for (int m = 16; m > 0; m /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
  if (lane == 0) fbuf[warp] = top;
  __syncthreads();
  top = fbuf[lane];
#pragma unroll
  for (int m = 16; m > 0; m /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
  __syncthreads();
  if (top == -INFINITY) {  // nothing can be drawn
    if (tid == 0) {
      a.tokens[b] = -1;
      if (a.logprobs) a.logprobs[b] = -INFINITY;
    }
    return;
  }
  float z = 0.0f;
  for (int64_t i = tid; i < V; i += kThreads) z += expf(logit(x, i) - top);
#pragma unroll
  for (int m = 16; m > 0; m /= 2) z += __shfl_xor_sync(0xffffffffu, z, m);
  if (lane == 0) fbuf[warp] = z;
  __syncthreads();
  z = fbuf[lane];
#pragma unroll
  for (int m = 16; m > 0; m /= 2) z += __shfl_xor_sync(0xffffffffu, z, m);

  const float t = a.temperature ? finite(a.temperature[b]) : 1.0f;
  const bool greedy = !(t >= 9.5367431640625e-7f);
  const float inv_t = greedy ? 1.0f : 1.0f / t;
  long long k = greedy ? 1 : (a.top_k ? a.top_k[b] : 0);
  if (k <= 0 || k > V) k = V;
  const float p = a.top_p ? a.top_p[b] : 1.0f;
  float min_p = a.min_p ? a.min_p[b] : 0.0f;
  min_p = min_p > 0.0f ? fminf(min_p, 1.0f) : 0.0f;

  // The kept prefix: keys above cut_key, and the first cut_ties of that key.
  uint32_t cut_key = 0;
  unsigned long long cut_ties = ~0ull;
  for (int by_weight = 0; by_weight < 2; ++by_weight) {
    unsigned long long want;  // the prefix ends where the running count / weight reaches this
    if (!by_weight) {
      if (k == V) continue;
      want = k;
    } else {
      if (!(p < 1.0f)) continue;
      unsigned long long sum = 0, tie = 0;
      for (int64_t i = tid; i < V; i += kThreads) {
        const float xi = logit(x, i);
        const uint32_t key = order_key(xi);
        if (key > cut_key) sum += weight(ratio(xi, top, inv_t));
        if (key == cut_key) tie = weight(ratio(xi, top, inv_t));
      }
      sum = block_sum(sum, buf);
      if (k < V) {  // ties at the top-k's last value all weigh the same
        __syncthreads();
        if (tid == 0) buf[0] = 0;
        __syncthreads();
        if (tie) buf[0] = tie;
        __syncthreads();
        tie = buf[0];
      }
      want = part_of(sum + (k < V ? cut_ties * tie : 0), (unsigned long long)(fmaxf(p, 0.0f) * 16777216.0f));
      if (want == 0) {
        cut_key = order_key(top);
        cut_ties = 1;
        continue;
      }
      if (want > sum) {  // the prefix ends among those ties
        cut_ties = (want - sum + tie - 1) / tie;
        continue;
      }
    }
    const uint32_t floor_key = by_weight ? cut_key : 0;
    uint32_t prefix = 0;
    unsigned long long before = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int64_t i = tid; i < V; i += kThreads) {
        const float xi = logit(x, i);
        const uint32_t key = order_key(xi);
        if (shift < 24 && (key >> (shift + 8)) != prefix) continue;
        if (key <= floor_key) continue;
        atomicAdd(&hist[key >> shift & 255], by_weight ? weight(ratio(xi, top, inv_t)) : 1ull);
      }
      __syncthreads();
      if (tid == 0) {
        int d = 255;
        unsigned long long run = before;
        while (d > 0 && run + hist[d] < want) run += hist[d--];
        pick_digit = d;
        pick_before = run;
      }
      __syncthreads();
      prefix = prefix << 8 | pick_digit;
      before = pick_before;
    }
    if (!by_weight) {
      cut_key = prefix;
      cut_ties = want - before;
    } else {
      // all of one value weigh the same: how many of them start under `want`
      unsigned long long w = 0;
      for (int64_t i = tid; i < V; i += kThreads)
        if (order_key(logit(x, i)) == prefix) w = weight(ratio(logit(x, i), top, inv_t));
      __syncthreads();
      if (tid == 0) buf[0] = 0;
      __syncthreads();
      if (w) buf[0] = w;
      __syncthreads();
      w = buf[0];
      cut_key = prefix;
      cut_ties = (want - before + w - 1) / w;
      __syncthreads();
    }
  }

  // The draw: each warp takes one stretch of the row.
  const int64_t seg = (V + 31) / 32, s0 = warp * seg, s1 = s0 + seg < V ? s0 + seg : V;
  unsigned long long ties = 0;
  for (int64_t i = s0 + lane; i < s1; i += 32) ties += order_key(logit(x, i)) == cut_key;
#pragma unroll
  for (int m = 16; m > 0; m /= 2) ties += __shfl_xor_sync(0xffffffffu, ties, m);
  __syncthreads();
  if (lane == 0) buf[warp] = ties;
  __syncthreads();
  unsigned long long ties0 = 0;
  for (int i = 0; i < warp; ++i) ties0 += buf[i];

  unsigned long long sum = 0, seen = ties0;
  for (int64_t i0 = s0; i0 < s1; i0 += 32) {
    const int64_t i = i0 + lane;
    const float xi = i < s1 ? logit(x, i) : -INFINITY;
    const uint32_t key = order_key(xi);
    const uint32_t same = __ballot_sync(0xffffffffu, i < s1 && key == cut_key);
    const unsigned long long nth = seen + __popc(same & ((1u << lane) - 1));
    const float e = ratio(xi, top, inv_t);
    if (i < s1 && (key > cut_key || (key == cut_key && nth < cut_ties)) && !(e < min_p)) sum += weight(e);
    seen += __popc(same);
  }
#pragma unroll
  for (int m = 16; m > 0; m /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  __syncthreads();
  if (lane == 0) buf[warp] = sum;
  __syncthreads();
  unsigned long long total = 0, run = 0;
  for (int i = 0; i < 32; ++i) {
    if (i < warp) run += buf[i];
    total += buf[i];
  }
  const float u = a.u[b];
  const unsigned long long share = u > 0.0f ? (unsigned long long)(fminf(u, 1.0f) * 16777216.0f) : 0ull;
  const unsigned long long r = part_of(total, share < 16777216ull ? share : 16777215ull);
  if (r < run || r >= run + sum) return;  // not in this warp's stretch
  seen = ties0;
  for (int64_t i0 = s0; i0 < s1; i0 += 32) {
    const int64_t i = i0 + lane;
    const float xi = i < s1 ? logit(x, i) : -INFINITY;
    const uint32_t key = order_key(xi);
    const uint32_t same = __ballot_sync(0xffffffffu, i < s1 && key == cut_key);
    const unsigned long long nth = seen + __popc(same & ((1u << lane) - 1));
    const float e = ratio(xi, top, inv_t);
    unsigned long long w =
        i < s1 && (key > cut_key || (key == cut_key && nth < cut_ties)) && !(e < min_p) ? weight(e) : 0;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
      const unsigned long long o = __shfl_up_sync(0xffffffffu, w, m);
      if (lane >= m) w += o;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, run + w > r);
    if (hit) {
      if (lane == __ffs(hit) - 1) {
        a.tokens[b] = i;
        if (a.logprobs) a.logprobs[b] = xi - top - logf(z);
      }
      return;
    }
    run += __shfl_sync(0xffffffffu, w, 31);
    seen += __popc(same);
  }
}

static_assert(sizeof(RowShared) % 16 == 0, "the row begins behind it, 16-byte aligned");
constexpr int kMaxSmem = (int)sizeof(RowShared) + kMaxRun * kThreads * 4;
static_assert(kMaxSmem <= 232448, "shared memory of a CTA");

// How many clusters of 4 or 8 CTAs run at once: fewer than the SMs hold CTAs, as a
// cluster stays within a group of SMs (36 and 15 on 152 SMs).  A CTA fills its SM's
// registers, so it does not depend on the row.
template <typename T>
int clusters_at_once(int C) {
  static std::atomic<int> known[64][2];
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  std::atomic<int> &was = known[dev & 63][C == 8];
  if ((n = was.load()) == 0) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = C;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(RowShared);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, sample_row_kernel<T>, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = 1;
    }
    was.store(n);
  }
  return n;
}

template <typename T>
int launch(const SampleArgs &a, cudaStream_t s) {
  cudaError_t e;
  if (a.V > (int64_t)8 * kMaxRun * kThreads) {
    // longer than a cluster holds: read again for every pass
    e = launch_pdl(sample_wide_kernel<T>, dim3((unsigned)a.B), dim3(kThreads), 0, s, a);
  } else {
    // As many CTAs a row as it needs.  More where the clusters run at once and the longer
    // joins pay (us, one row of 50272: drawn freely 14.4 on one CTA, 11.5 on 8; top-p 33.7,
    // 30.6; top-k 17.7, 19.8; of 8000: 8.3, 10.4; 22.6, 26.7; 13.1, 19.3; of 200000, on 4
    // and on 8: 17.7, 13.8; 50, 47; 23.5, 21.4.  16 rows of 50272 on 8, two turns: 22; 60; 39.)
    int C = 1;
    while ((int64_t)C * kMaxRun * kThreads < a.V) C *= 2;
    if (C > 1 || (!a.top_k && a.V > (int64_t)kMaxRun / 2 * kThreads))
      for (int more = 8; more >= 4; more /= 2)
        if (more > C && a.B <= clusters_at_once<T>(more)) {
          C = more;
          break;
        }
    const int R = (int)((a.V + (int64_t)C * kThreads - 1) / ((int64_t)C * kThreads)) | 1;
    const size_t smem = sizeof(RowShared) + (size_t)R * kThreads * sizeof(float);
    if (a.B * C > 0x7fffffff) return set_error(TP_ERR_UNSUPPORTED, "too many rows for one launch");
    auto kern = sample_row_kernel<T>;
    // The limit belongs to the function, not to this call: always the largest, so that a thread
    // with shorter rows does not lower it between another's setting and launch.
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return cuda_error(e, "sample launch");
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)(a.B * C));
    cfg.blockDim = dim3(kThreads);
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
    const bool reorder = a.B * C > sm_count() && (a.top_k || a.top_p);
    e = cudaLaunchKernelEx(&cfg, kern, a, C, R, reorder);
  }
  if (e != cudaSuccess) return cuda_error(e, "sample launch");
  note_launch();
  return TP_OK;
}

}  // namespace

int launch_sample(const SampleArgs &a, cudaStream_t s) {
  if (a.in_dt == TP_F32) return launch<float>(a, s);
  return a.in_dt == TP_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

}  // namespace tp
