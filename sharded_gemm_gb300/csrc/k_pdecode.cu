// k_pdecode.cu -- tp_paged_decode: attention of one token per sequence over the
// paged cache, split evenly over the GPU and joined in a fixed order.
//
// Work.  An item is one sequence, rank, key-value head and group of at most
// 8 * NT query heads of it.  Its visible positions are cut into units of 128
// (eight chunks of 16); the units of all items, in order, are dealt out to the
// CTAs in consecutive ranges of equal cost (kUnitCost a unit, kItemCost an item:
// its warps' parts have to be merged), so every SM has the same work however
// uneven the lengths are.  A CTA's range covers pieces of one or more items; an
// item that spans CTAs leaves its pieces' unnormalised sums in the workspace and
// the last CTA to arrive joins them in CTA order (same bytes every time).
//
// A piece.  Warp w takes chunks w, w + 8, ... through a ring of asynchronous
// copies of its own (no barrier between warps until the piece ends); chunk rows
// that hold no visible position arrive as zeros without being read, so stale
// rows (NaN too) reach neither product.  Per chunk, with S^T = K Q^T (16
// positions x heads, positions as the rows so that up to 8 heads cost one
// product) and O^T += V^T P^T:
//   the running maximum is raised only where a score passes it by more than 2^8
//   in the exponential (a warp vote per chunk in place of a cross-lane maximum);
//   the sums stay per lane until the piece ends.
// The maximum is a score that occurs (or is within 2^8 of one), so float16
// terms lose nothing to their range.
//
// Bytes bound it: every visible key and value is read once.  Measured against the
// copy rate (6.79 TB/s): 64 sequences of 1000..16384, 8 heads on one of 128, 333 us
// (101%); 16 of 100..4096 with as many key as query heads 93 us (96%); 48 windows of
// 1024 on heads of 64, capped, 26 to 28 us (50%: 4 us to the first bytes, then about 3 us
// a piece besides its units, of which a CTA has 20 in 3.1 pieces); one sequence of 517 8.9 us, a chain of latencies.  The softmax's terms
// are rounded to the 16-bit type for the second product, as its operands are.
#include "mma16.cuh"

namespace tp {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kUnit = 16 * kWarps;
constexpr float kSlack = 8.0f;  // how far (log2) a score may pass the running maximum

template <int D, int NT>
struct Shape {
  static constexpr int kChunkBytes = 16 * D * 2;                     // K or V of one chunk
  static constexpr int kStages = (NT == 1 ? 24576 : 16384) / (2 * kChunkBytes);
  static constexpr int kHeads = 8 * NT;
  static constexpr int kRow = D + 4;                                  // floats of a merged head's row
  static constexpr int kRingBytes = kWarps * kStages * 2 * kChunkBytes;
  static constexpr int kMergeBytes = kWarps * kHeads * (kRow + 2) * 4;
  static constexpr int kSmem = kRingBytes + kMergeBytes;
  static constexpr int kSlot = kHeads * (D + 2);                      // floats of a workspace piece
  // Cost of a unit and of an item (its start and the merge of its parts), in
  // 0.37 us: a unit streams in 0.73 us at D = 64 and 1.47 at 128.  Item costs of
  // 3, 4, 5, 6, 8 and 10 gave 98, 95, 94, 93, 92 and 92 us for 16 sequences of
  // 100..4096 positions on 32 heads of 128, and 31, 27.2, 26.5, 25.8, 25.4 and 25.4
  // for 48 windows of 1024 at 64.
  static constexpr int kUnitCost = D / 32, kItemCost = 8;
};

struct Plan {
  int items_per_seq, groups;  // items of a sequence; head groups of a key-value head
  float *ws;
  int *counters;
};

// Where the visible positions of a sequence begin (rounded down to a chunk) and end.
struct Span {
  int first, from, to, units;
};
__device__ __forceinline__ Span span_of(const AttnArgs &a, int64_t b) {
  Span s;
  int64_t n = a.seq_lens[b];
  if (n < 0 || n > a.cap) {
    record_bad_value(a.status);
    n = n < 0 ? 0 : a.cap;
  }
  s.to = (int)n;
  s.first = a.window && s.to > a.window ? s.to - a.window : 0;
  s.from = s.first & ~15;
  s.units = (s.to - s.from + kUnit - 1) / kUnit;
  return s;
}

// a / b, both positive; 64-bit divisions only where 32 bits do not hold the numbers.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (a | b) >> 32 ? a / b : (uint32_t)a / (uint32_t)b;
}

// A place in the CTA's list of pieces.
struct Piece {
  int64_t b;
  int item, unit0, units;  // item of sequence b, the piece's first unit in it, its units
  long long at;            // where the item begins, in cost
  Span span;
  bool valid;
};

// An item of which this CTA has left a piece in the workspace: CTAs c0 .. c1 share it.
struct Join {
  long long c0, c1;
  int64_t out;  // of its first head, in o[r]
  int r, heads;
  int last;     // this CTA came last, and joins
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ AttnArgs a, const Plan plan) {
  using Sh = Shape<D, NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ long long s_scan[kWarps + 1];
  __shared__ long long s_b[2], s_at[2];
  __shared__ Join s_join;
  __shared__ Piece s_first;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  griddep_launch_dependents();
  griddep_wait();

  // ---- this CTA's range of units
  const int ips = plan.items_per_seq;
  const int64_t per = (a.B + kThreads - 1) / kThreads, b0 = tid * per, b1 = b0 + per < a.B ? b0 + per : a.B;
  long long mine = 0;
  constexpr int UC = Sh::kUnitCost, IC = Sh::kItemCost;
  auto cost = [&](const Span &s) { return s.units ? ips * (IC + (long long)UC * s.units) : 0ll; };
  for (int64_t b = b0; b < b1; ++b) mine += cost(span_of(a, b));
  long long scan = mine;
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    const long long o = __shfl_up_sync(0xffffffffu, scan, m);
    if (lane >= m) scan += o;
  }
  if (lane == 31) s_scan[warp] = scan;
  __syncthreads();
  long long before = scan - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  // every CTA's range is at least a unit long: those inside an item then hold a unit of it
  const long long even = quotient(total + gridDim.x - 1, gridDim.x), share = even > UC ? even : UC, cta = blockIdx.x;
  const long long x0 = cta * share < total ? cta * share : total, x1 = x0 + share < total ? x0 + share : total;
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // the sequences that hold the range's first and last place
    const long long x = i ? x1 - 1 : x0;
    if (x0 < x1 && x >= before && x < before + mine) {
      long long at = before;
      for (int64_t b = b0; b < b1; ++b) {
        const long long c = cost(span_of(a, b));
        if (x < at + c) {
          s_b[i] = b;
          s_at[i] = at;
          break;
        }
        at += c;
      }
    }
  }
  __syncthreads();

  // ---- the list of pieces, walked twice: by the copies, ahead, and by the products.
  // Unit u of an item that begins at `at` belongs to the CTA whose range holds
  // at + IC + u * UC.  Where the last item goes on in the next CTA its piece is taken
  // first, so that the join with the others' has the rest of the range to hide under
  // (16 sequences of 100..4096: 91.9 us; taken last, 93.5; 48 windows 25.4 and 25.2).
  long long stop = x1;
  auto cut = [&](Piece &p) {  // p is an item: its units in this range
    const long long lo = x0 - p.at - IC + UC - 1, hi = x1 - p.at - IC + UC - 1;
    p.unit0 = lo > 0 ? (int)(lo / UC) : 0;
    const int end = hi > 0 ? (hi / UC < p.span.units ? (int)(hi / UC) : p.span.units) : 0;
    p.units = end - p.unit0;
  };
  auto settle = [&](Piece &p) {  // p is an item: its units in this range, or the next item that has some
    for (;;) {
      if (p.at >= stop) {
        p.valid = false;
        return;
      }
      cut(p);
      if (p.units > 0) return;
      p.at += IC + (long long)UC * p.span.units;
      if (++p.item == ips) {
        p.item = 0;
        do {
          if (++p.b >= a.B) {
            p.valid = false;
            return;
          }
          p.span = span_of(a, p.b);
        } while (p.span.units == 0);
      }
    }
  };
  auto item_at = [&](Piece &p, int i, long long x) {  // the item that holds place x, in sequence s_b[i]
    p.b = s_b[i];
    p.span = span_of(a, p.b);
    const long long each = IC + (long long)UC * p.span.units;
    p.item = (int)quotient(x - s_at[i], each);
    p.at = s_at[i] + p.item * each;
  };
  Piece p;
  p.valid = x0 < x1;
  if (p.valid) {
    item_at(p, 0, x0);
    settle(p);
    if (tid == 0) s_first = p;
    if (p.valid && p.at + IC + (long long)UC * p.span.units < x1) {  // it goes on behind p
      Piece last;
      last.valid = true;
      item_at(last, 1, x1 - 1);
      cut(last);
      if (last.units > 0 && last.unit0 + last.units < last.span.units) stop = last.at, p = last;
    }
    __syncthreads();  // s_first
  }
  auto next_piece = [&](Piece &p) {
    if (p.at >= stop) {
      p = s_first;
      return;
    }
    p.at += IC + (long long)UC * p.span.units;
    if (++p.item == ips) {
      p.item = 0;
      do {
        if (++p.b >= a.B) {
          p.valid = false;
          return;
        }
        p.span = span_of(a, p.b);
      } while (p.span.units == 0);
    }
    settle(p);
  };

  const uint32_t ring = smem_u32(smem) + warp * (Sh::kStages * 2 * Sh::kChunkBytes);
  float *merge = reinterpret_cast<float *>(smem + Sh::kRingBytes);

  // ---- copies
  Piece cp = p;
  int cp_unit = 0, cp_stage = 0, cp_page_at = -32;
  int cp_pages = 0;  // lane i: the page of this warp's chunk in unit cp_page_at + i
  constexpr int kLanesPerRow = D / 8, kRowsPerCopy = 32 / kLanesPerRow;
  const int c_row = lane / kLanesPerRow, c_col = lane % kLanesPerRow;
  const T *cp_k = nullptr, *cp_v = nullptr;  // the piece's head in page 0, at this lane's place
  auto cp_head = [&]() {
    const int rh = cp.item / plan.groups, r = rh / a.Hk, h = rh - r * a.Hk;
    const int64_t off = ((int64_t)h * a.page + c_row) * D + c_col * 8;
    cp_k = static_cast<const T *>(a.k_cache[r]) + off, cp_v = static_cast<const T *>(a.v_cache[r]) + off;
  };
  if (cp.valid) cp_head();
  auto issue = [&]() {
    if (cp.valid) {
      const int j0 = cp.span.from + (cp.unit0 + cp_unit) * kUnit + warp * 16;
      if (cp_unit - cp_page_at >= 32) {
        cp_page_at = cp_unit;
        const int j = j0 + lane * kUnit;
        cp_pages = -1;
        if (cp_unit + lane < cp.units && j < cp.span.to) {
          cp_pages = a.block_table[cp.b * a.ld_table + (j >> a.page_log2)];
          if (cp_pages < 0 || cp_pages >= a.pages) {
            record_bad_value(a.status);
            cp_pages = -1;
          }
        }
      }
      const int pg = __shfl_sync(0xffffffffu, cp_pages, cp_unit - cp_page_at);
      const int64_t base = (int64_t)(pg < 0 ? 0 : pg) * a.ld_page + (j0 & (a.page - 1)) * D;
      const T *k = cp_k + base, *v = cp_v + base;
      // visible rows of the chunk, from this lane's first
      const int lo = cp.span.first - j0 - c_row, hi = pg < 0 ? -1 : cp.span.to - j0 - c_row;
      const uint32_t dst = ring + cp_stage * (2 * Sh::kChunkBytes) + c_row * (D * 2);
#pragma unroll
      for (int i = 0; i < 16 / kRowsPerCopy; ++i) {
        const int row = i * kRowsPerCopy;
        const bool ok = row >= lo && row < hi;
        const uint32_t off = row * (D * 2) + ((c_col ^ ((row + c_row) & 7)) << 4);
        cp_async16(dst + off, k + row * D, ok);
        cp_async16(dst + Sh::kChunkBytes + off, v + row * D, ok);
      }
      if (++cp_unit == cp.units) {
        next_piece(cp);
        if (cp.valid) cp_head();
        cp_unit = 0;
        cp_page_at = -32;
      }
    }
    cp_async_commit();
    cp_stage = cp_stage + 1 == Sh::kStages ? 0 : cp_stage + 1;
  };
#pragma unroll
  for (int i = 0; i < Sh::kStages - 1; ++i) issue();

  // ---- products
  const float to_log2 = 1.4426950408889634f;
  const float qk_scale = a.softcap > 0.0f ? a.scale / a.softcap * 2.0f * to_log2 : a.scale * to_log2;
  const float cap_log2 = a.softcap * to_log2;
  int stage = 0;
  const int G = a.Hq / a.Hk;
  // A piece left in the workspace is joined with the others' at the end of the next piece:
  // until then one warp waits for the count of those that came, not the CTA (2 to 3 us of
  // round trips; 48 windows of 1024 took 1.0 us longer).
  bool joins = false;
  auto join = [&]() {
    const long long c0 = s_join.c0, c1 = s_join.c1;
    if (!s_join.last) return;
    if (tid == 0) plan.counters[c0] = 0;  // ready for the next call
    for (int e = tid; e < s_join.heads * D; e += kThreads) {
      const int head = e / D, d = e % D;
      float top = -INFINITY, sum = 0.0f, acc = 0.0f;
      for (long long c = c0; c <= c1; c += 8) {  // eight pieces' loads at a time
        float mc[8], lc[8], oc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float *s = plan.ws + ((c + i) * 2 + (c + i == c0 ? 1 : 0)) * Sh::kSlot;
          const bool is = c + i <= c1;
          mc[i] = is ? __ldcg(s + Sh::kHeads * D + head) : -INFINITY;
          lc[i] = is ? __ldcg(s + Sh::kHeads * (D + 1) + head) : 0.0f;
          oc[i] = is ? __ldcg(s + head * D + d) : 0.0f;
        }
        float tn = top;
#pragma unroll
        for (int i = 0; i < 8; ++i) tn = fmaxf(tn, mc[i]);
        const float mm = tn == -INFINITY ? 0.0f : tn, f0 = exp2f(top - mm);
        sum *= f0, acc *= f0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float f1 = exp2f(mc[i] - mm);
          sum += f1 * lc[i];
          acc += f1 * oc[i];
        }
        top = tn;
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      static_cast<T *>(a.o[s_join.r])[s_join.out + head * D + d] = static_cast<T>(acc * inv);
    }
  };
  while (p.valid) {
    const int rh = p.item / plan.groups, grp = p.item - rh * plan.groups, r = rh / a.Hk, h = rh - r * a.Hk;
    const int heads = G - grp * Sh::kHeads < Sh::kHeads ? G - grp * Sh::kHeads : Sh::kHeads;
    const int64_t head0 = (int64_t)h * G + grp * Sh::kHeads;
    // Q^T fragments: head g of each group of eight, pairs of values
    uint32_t q[NT][D / 16][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool has = n * 8 + g < heads;
      const uint16_t *row =
          static_cast<const uint16_t *>(a.q[r]) + p.b * a.ldq + (head0 + (has ? n * 8 + g : 0)) * D + 2 * t;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint16_t *e = row + ks * 16 + i * 8;
          q[n][ks][i] = has ? (uint32_t)__ldg(e) | (uint32_t)__ldg(e + 1) << 16 : 0u;
        }
    }
    float m[NT][2], l[NT][2], o[NT][D / 16][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
    }

    for (int unit = 0; unit < p.units; ++unit) {
      cp_async_wait<Sh::kStages - 2>();
      __syncwarp();
      issue();
      const uint32_t kbase = ring + stage * (2 * Sh::kChunkBytes), vbase = kbase + Sh::kChunkBytes;
      stage = stage + 1 == Sh::kStages ? 0 : stage + 1;
      const int j0 = p.span.from + (p.unit0 + unit) * kUnit + warp * 16;
      if (j0 >= p.span.to) continue;

      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
      {
        const int row = lane & 15, hi = lane >> 4;  // matrices: rows 0-7, 8-15, then the next 8 values
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t ka[4];
          ldmatrix4(kbase + row * (D * 2) + (((2 * ks + hi) ^ (row & 7)) << 4), ka);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816<T>(s[n], ka, q[n][ks][0], q[n][ks][1]);
        }
      }
      // scores in units of log2
      const int lo = p.span.first - j0, hi = p.span.to - j0;  // visible rows [lo, hi)
      const bool edge = lo > 0 || hi < 16;
      bool rise = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = s[n][i] * qk_scale;
          if (a.softcap > 0.0f) x = capped(x, cap_log2);  // (tanhf and exp2f: 2.2 us of 31)
          if (edge) {
            const int row = g + (i & 2) * 4;
            if (row < lo || row >= hi) x = -INFINITY;
          }
          s[n][i] = x;
          rise |= x > m[n][i & 1] + kSlack;
        }
      if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = fmaxf(s[n][c], s[n][c + 2]);
#pragma unroll
            for (int x = 4; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            if (top > m[n][c]) {  // the same in all lanes of a head
              const float keep = exp2_approx(m[n][c] - top);
              m[n][c] = top;
              l[n][c] *= keep;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) o[n][i][c] *= keep, o[n][i][c + 2] *= keep;
            }
          }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float mm = m[n][i & 1];
          e[i] = exp2_approx(s[n][i] - (mm == -INFINITY ? 0.0f : mm));
        }
        l[n][0] += e[0] + e[2];
        l[n][1] += e[1] + e[3];
        pb[n][0] = movmatrix_trans(Half2<T>::pack(e[0], e[1]));
        pb[n][1] = movmatrix_trans(Half2<T>::pack(e[2], e[3]));
      }
      {
        const int row = (lane & 7) + ((lane >> 4) << 3), hi8 = (lane >> 3) & 1;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t va[4];  // V^T: 16 values x 16 positions
          ldmatrix4_trans(vbase + row * (D * 2) + (((2 * i + hi8) ^ (row & 7)) << 4), va);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816<T>(o[n][i], va, pb[n][0], pb[n][1]);
        }
      }
    }

    // ---- the eight warps' parts of the piece
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], x);
        const int head = n * 8 + 2 * t + c;
        if (head < heads) {
          float *row = merge + (warp * Sh::kHeads + head) * Sh::kRow;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) row[i * 16 + g] = o[n][i][c], row[i * 16 + g + 8] = o[n][i][c + 2];
          if (g == 0) {
            float *ml = merge + kWarps * Sh::kHeads * Sh::kRow;
            ml[warp * Sh::kHeads + head] = m[n][c];
            ml[(kWarps + warp) * Sh::kHeads + head] = l[n][c];
          }
        }
      }
    __syncthreads();
    if (joins) join();
    joins = false;
    const bool whole = p.units == p.span.units;
    float *slot = plan.ws + (cta * 2 + (p.unit0 == 0 ? 1 : 0)) * Sh::kSlot;  // an item begins, or goes on, here
    const float *ml = merge + kWarps * Sh::kHeads * Sh::kRow;
    for (int e = tid; e < heads * D; e += kThreads) {
      const int head = e / D, d = e % D;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * Sh::kHeads + head]);
      const float mm = top == -INFINITY ? 0.0f : top;
      float sum = 0.0f, acc = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(ml[w * Sh::kHeads + head] - mm);
        sum += f * ml[(kWarps + w) * Sh::kHeads + head];
        acc += f * merge[(w * Sh::kHeads + head) * Sh::kRow + d];
      }
      if (whole) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        static_cast<T *>(a.o[r])[p.b * a.ldo + (head0 + head) * D + d] = static_cast<T>(acc * inv);
      } else {
        slot[head * D + d] = acc;
        if (d == 0) slot[Sh::kHeads * D + head] = top, slot[Sh::kHeads * (D + 1) + head] = sum;
      }
    }
    __syncthreads();  // the merge rows are free again, and the piece is written
    if (!whole) {
      if (tid == 0) {
        // the CTAs of this item, by the places of its first and last unit
        const long long f = p.at + IC, e0 = f + (long long)UC * (p.span.units - 1);
        s_join.c0 = quotient(f, share), s_join.c1 = quotient(e0, share);
        s_join.out = p.b * a.ldo + head0 * D;
        s_join.r = r, s_join.heads = heads;
        // releases the CTA's parts (the barrier orders the other threads' before it), and
        // acquires those of the CTAs counted before
        int came;
        asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                     : "=r"(came)
                     : "l"(plan.counters + s_join.c0)
                     : "memory");
        s_join.last = came == (int)(s_join.c1 - s_join.c0);
      }
      joins = true;
    }
    next_piece(p);
  }
  if (joins) {
    __syncthreads();
    join();
  }
  cp_async_wait<0>();

  // Sequences with nothing visible: zeros.
  for (int64_t b = cta; b < a.B; b += gridDim.x)
    if (span_of(a, b).units == 0)
      for (int i = tid; i < a.N * a.Hq * D; i += kThreads)
        static_cast<T *>(a.o[i / (a.Hq * D)])[b * a.ldo + i % (a.Hq * D)] = static_cast<T>(0.0f);
}

template <typename T, int D, int NT>
int launch(const AttnArgs &a, cudaStream_t s) {
  using Sh = Shape<D, NT>;
  static_assert(Sh::kSmem + 1024 <= 232448, "shared memory of a CTA");
  Plan plan;
  const int G = a.Hq / a.Hk;
  plan.groups = (G + Sh::kHeads - 1) / Sh::kHeads;
  plan.items_per_seq = a.N * a.Hk * plan.groups;
  const int grid = sm_count();
  if (int rc = split_workspace(s, (size_t)grid * 2 * Sh::kSlot * sizeof(float), grid, &plan.ws, &plan.counters))
    return rc;
  auto kern = decode_kernel<T, D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
  if (e == cudaSuccess) e = launch_pdl(kern, dim3(grid), dim3(kThreads), Sh::kSmem, s, a, plan);
  if (e != cudaSuccess) return cuda_error(e, "decode launch");
  note_launch();
  return TP_OK;
}

template <typename T>
int launch_t(const AttnArgs &a, cudaStream_t s) {
  const bool one = a.Hq / a.Hk <= 8;
  if (a.D == 64) return one ? launch<T, 64, 1>(a, s) : launch<T, 64, 2>(a, s);
  return one ? launch<T, 128, 1>(a, s) : launch<T, 128, 2>(a, s);
}

}  // namespace

int launch_decode(const AttnArgs &a, cudaStream_t s) {
  return a.dt == TP_BF16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<__half>(a, s);
}

}  // namespace tp
