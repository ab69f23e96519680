// k_plan.cu -- tp_paged_plan and tp_lora_plan: what a serving step needs to know of its
// tokens, built from the requests' lengths on the GPU.
//
// tp_paged_plan.  Three running sums over the sequences (tokens, pages that ended ones
// give back, pages needed) place everything: token i of sequence b in row cu[b] + i, the
// i-th page given back on top of the pool, the i-th page needed taken from the top.  One
// CTA takes the sums; a barrier lies between its last read of what the outputs may be and
// the first write.  Then pages given back, pages taken and rows are dealt to its threads,
// each of which finds its sequence by bisection of the sums in shared memory and needs
// nothing that another thread has just written.  The rows of a large step are a second
// kernel's.
//
// tp_lora_plan.  A stable counting sort by adapter: tokens of each adapter counted in
// shared memory, their running sum, and then one warp walks the sequences in order, 32 at
// a time, and gives each the place behind the earlier ones of its adapter.  The tokens are
// then dealt to all threads.  Of a large step's several CTAs each does the counting for
// itself.
//
// Both are bound by latency: two or three dependent loads, the sums' barriers, the
// bisections.  Measured: 4 sequences 3.3 us; 256 of 1 to 8 tokens 5, 10 with 13000 pages given
// back, and 7 for their adapters' plan; 96 prompts of 106000 rows 13 with both.
#include "ptx.cuh"
#include "serve.cuh"

namespace tp {
namespace {

constexpr int kThreads = 1024;

// Sums of lower threads over the block of N values; `total` the sums of all.  buf: 32 N.
template <int N>
__device__ __forceinline__ void scan_before(int64_t (&v)[N], int64_t (&total)[N], int64_t *buf) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int64_t run[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    run[i] = v[i];
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
      const int64_t o = __shfl_up_sync(0xffffffffu, run[i], m);
      if (lane >= m) run[i] += o;
    }
    if (lane == 31) buf[i * 32 + warp] = run[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t w = buf[i * 32 + lane];
    int64_t base = lane < warp ? w : 0, all = w;
#pragma unroll
    for (int m = 16; m > 0; m /= 2) {
      base += __shfl_xor_sync(0xffffffffu, base, m);
      all += __shfl_xor_sync(0xffffffffu, all, m);
    }
    v[i] = base + run[i] - v[i];
    total[i] = all;
  }
}

// The last b of 0..n-1 with sums[b] <= at; sums ascends from 0 and at >= 0.
__device__ __forceinline__ int holder(const int32_t *sums, int n, int32_t at) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (sums[mid] <= at) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Rows that one CTA takes itself.  (Four turns of its threads, 3 us; a second launch costs 2.)
constexpr int64_t kOwnRows = 4096;

__global__ void __launch_bounds__(kThreads) plan_kernel(const __grid_constant__ PlanArgs a) {
  extern __shared__ int32_t smem[];
  __shared__ int64_t buf[96];
  const int B = (int)a.B, tid = threadIdx.x;
  int32_t *cu = smem, *need_at = cu + B, *back_at = need_at + B, *after = back_at + B, *held = after + B;
  griddep_launch_dependents();
  griddep_wait();

  // ---- a run of sequences a thread, and the sums before them
  struct Sequence {
    int64_t tokens, need, back, end, own, len;
    bool ok;
  };
  const int64_t page = 1ll << a.page_log2;
  auto sequence = [&](int b) {
    const int64_t c = a.counts[b], less = a.rejected ? a.rejected[b] : 0;
    Sequence s{0, 0, 0, 0, a.owned[b], a.seq_lens[b], false};
    const bool held = s.own >= 0 && s.own <= a.width;
    if (c < 0) {
      s.ok = held;
      if (held) s.back = s.own;
      return s;
    }
    s.end = s.len - less + c, s.tokens = c;
    const int64_t pages = (s.end + page - 1) >> a.page_log2;
    s.need = pages > s.own ? pages - s.own : 0;
    s.ok = held && s.len >= 0 && less >= 0 && less <= s.len && s.end <= a.cap && (s.own << a.page_log2) >= s.len - less;
    return s;
  };
  const int64_t F = a.free_count[0];
  const int run = (B + kThreads - 1) / kThreads, b0 = tid * run, b1 = min(b0 + run, B);
  bool bad = F < 0 || F > a.pages;
  int64_t sums[3] = {0, 0, 0}, total[3];
  Sequence only{0, 0, 0, 0, 0, 0, true};  // of a run of one
  for (int b = b0; b < b1; ++b) {
    only = sequence(b);
    if (only.ok) sums[0] += only.tokens, sums[1] += only.need, sums[2] += only.back;
    else bad = true;
  }
  scan_before<3>(sums, total, buf);
  const int64_t top = F + total[2];  // of the pool, what ended sequences give back on it
  bad = __syncthreads_or(bad) || top > a.pages || total[0] > a.T;
  const bool fits = !bad && total[1] <= top;
  for (int b = b0; b < b1; ++b) {
    if (run > 1) only = sequence(b);
    cu[b] = fits ? (int32_t)sums[0] : 0, need_at[b] = (int32_t)sums[1], back_at[b] = (int32_t)sums[2];
    after[b] = (int32_t)(fits ? only.end : only.len), held[b] = (int32_t)only.own;  // or an empty step
    sums[0] += only.tokens, sums[1] += only.need, sums[2] += only.back;
  }
  __syncthreads();  // all is read that is written below, and the sums are in shared memory

  const int total_tokens = fits ? (int)total[0] : 0, total_need = fits ? (int)total[1] : 0;
  const int total_back = fits ? (int)total[2] : 0;
  for (int b = tid; b < B; b += kThreads) {
    const int all = b + 1 < B ? need_at[b + 1] : (int)total[1];
    const bool ends = fits && (b + 1 < B ? back_at[b + 1] : total_back) > back_at[b];
    a.cu[b] = cu[b];
    a.new_lens[b] = after[b];
    // (a sequence that ended with no pages has none to need either)
    a.new_owned[b] = !fits ? held[b] : ends ? 0 : held[b] + (all - need_at[b]);
  }
  if (tid == 0) {
    a.cu[B] = total_tokens;
    a.new_free_count[0] = fits ? (int32_t)(top - total[1]) : (int32_t)F;
    a.missing[0] = bad ? -1 : fits ? 0 : (int32_t)(total[1] - top);
    if (bad) record_bad_value(a.status);
  }
  // ---- pages given back go on top of the pool, and what is needed is taken from there
  // The sequence of the i-th of `sums`' pages, asked for i after i: found anew behind its end.
  struct Walk {
    int b = 0, end = 0;
    __device__ __forceinline__ int at(const int32_t *sums, int n, int all, int i) {
      if (i >= end) {
        b = holder(sums, n, i);
        end = b + 1 < n ? sums[b + 1] : all;
      }
      return b;
    }
  };
  auto given = [&](int i, int b) { return a.table[b * a.ld_table + (i - back_at[b])]; };
  auto taken = [&](int i) {
    const int64_t at = top - 1 - i;
    return at < F ? a.free_pages[at] : given((int)(at - F), holder(back_at, B, (int)(at - F)));
  };
  // 256 pages a warp at a time, the last warp first (the first have the tokens): a lane's
  // eight are mostly of one sequence, which takes one bisection, and under one latency.
  // (13000 pages given back one by one: 15 us, all of it bisections.)
  const int warp = kThreads / 32 - 1 - tid / 32, lane = tid % 32;
  for (int i0 = warp * 256 + lane; i0 < total_back; i0 += 8 * kThreads) {
    Walk w;
    int32_t v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u * 32;
      if (i < total_back) v[u] = given(i, w.at(back_at, B, total_back, i));
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i0 + u * 32 < total_back) a.free_pages[F + i0 + u * 32] = v[u];
  }
  for (int i0 = warp * 128 + lane; i0 < total_need; i0 += 4 * kThreads) {
    Walk w;
    int32_t v[4];
    int64_t to[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * 32;
      if (i >= total_need) continue;
      const int b = w.at(need_at, B, total_need, i);
      to[u] = b * a.ld_table + held[b] + (i - need_at[b]);
      v[u] = taken(i);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * 32 < total_need) a.table[to[u]] = v[u];
  }
  // ---- the tokens
  if (a.T > kOwnRows) return;
  for (int t = tid; t < a.T; t += kThreads) {
    int32_t position = 0;
    int64_t slot = -1;
    if (t < total_tokens) {
      const int b = holder(cu, B, t), end = b + 1 < B ? cu[b + 1] : total_tokens;
      position = after[b] - (end - t);
      const int j = position >> a.page_log2;
      const int32_t p = j < held[b] ? a.table[b * a.ld_table + j] : taken(need_at[b] + j - held[b]);
      if (p >= 0 && p < a.pages) slot = ((int64_t)p << a.page_log2) + (position & (int)(page - 1));
      else record_bad_value(a.status);
    }
    a.positions[t] = position;
    a.slots[t] = slot;
  }
}

// The rows of a large step, from what plan_kernel wrote.
__global__ void __launch_bounds__(512) plan_rows_kernel(const __grid_constant__ PlanArgs a) {
  extern __shared__ int32_t cu[];
  const int B = (int)a.B, tid = threadIdx.x;
  griddep_wait();
  for (int b = tid; b <= B; b += 512) cu[b] = a.cu[b];
  __syncthreads();
  const int total = cu[B];
  for (int64_t t = blockIdx.x * 512ll + tid; t < a.T; t += gridDim.x * 512ll) {
    int32_t position = 0;
    int64_t slot = -1;
    if (t < total) {
      const int b = holder(cu, B, (int)t);
      position = a.new_lens[b] - (cu[b + 1] - (int)t);
      const int32_t p = a.table[b * a.ld_table + (position >> a.page_log2)];
      if (p >= 0 && p < a.pages) slot = ((int64_t)p << a.page_log2) + (position & ((1 << a.page_log2) - 1));
      else record_bad_value(a.status);
    }
    a.positions[t] = position;
    a.slots[t] = slot;
  }
}

__global__ void __launch_bounds__(kThreads) group_kernel(const __grid_constant__ GroupArgs a) {
  extern __shared__ int32_t smem[];
  __shared__ int64_t buf[64];
  const int B = (int)a.B, n = (int)a.n, tid = threadIdx.x, lane = tid % 32;
  int32_t *cu = smem, *first = cu + B + 1, *tokens = first + B;  // (B + 1), (B), (n + 1)
  griddep_launch_dependents();
  griddep_wait();
  for (int b = tid; b <= B; b += kThreads) cu[b] = a.cu ? a.cu[b] : b;
  for (int i = tid; i <= n; i += kThreads) tokens[i] = 0;
  __syncthreads();
  // adapter n: none
  auto adapter = [&](int b) {
    const int id = a.adapters[b];
    return id < 0 || id >= n ? n : id;
  };
  bool bad = false;
  for (int b = tid; b < B; b += kThreads) {
    const int r0 = cu[b], r1 = cu[b + 1];
    if (r0 < 0 || r1 < r0 || r1 > a.T || (b == 0 && r0 != 0)) bad = true;
    else if (r1 > r0) atomicAdd(&tokens[adapter(b)], r1 - r0);
    if (a.adapters[b] >= n) record_bad_value(a.status);
  }
  bad = __syncthreads_or(bad);
  // ---- a run of adapters a thread: the places and groups before them
  const int run = (n + kThreads) / kThreads, i0 = min(tid * run, n + 1), i1 = min(i0 + run, n + 1);
  int64_t sums[2] = {0, 0}, total[2];
  for (int i = i0; i < i1; ++i) sums[0] += tokens[i], sums[1] += tokens[i] > 0;
  scan_before<2>(sums, total, buf);
  const int all = bad ? 0 : (int)total[0], groups = bad ? 0 : (int)total[1];
  int4 *out = reinterpret_cast<int4 *>(a.plan + 4);
  int without = 0;
  for (int i = i0; i < i1; ++i) {
    const int count = tokens[i];
    if (count > 0 && !bad && blockIdx.x == 0)
      out[sums[1]] = make_int4(i < n ? i : -1, (int)sums[0], count, 0);
    if (i == n) without = count;
    tokens[i] = (int)sums[0];  // where the adapter's next sequence goes
    sums[0] += count, sums[1] += count > 0;
  }
  if (blockIdx.x == 0) {
    for (int64_t i = groups + tid; i < a.most; i += kThreads) out[i] = make_int4(-1, -1, -1, -1);
    if (i0 <= n && n < i1)
      *reinterpret_cast<int4 *>(a.plan) = make_int4(groups, bad ? 0 : all - without, 0, 0);
    if (bad && tid == 0) record_bad_value(a.status);
  }
  __syncthreads();
  // ---- the sequences in order, 32 at a time
  if (tid < 32 && !bad) {
    for (int base = 0; base < B; base += 32) {
      const int b = base + lane, len = b < B ? cu[b + 1] - cu[b] : 0, id = b < B ? adapter(b) : n + 1 + lane;
      const uint32_t peers = __match_any_sync(0xffffffffu, id);
      const int most = __reduce_max_sync(0xffffffffu, __popc(peers));
      int before = 0, mine = 0;
      uint32_t rest = peers;
      for (int i = 0; i < most; ++i) {  // each lane its own peers, one after the other
        const int from = rest ? __ffs(rest) - 1 : lane;
        const int l = __shfl_sync(0xffffffffu, len, from);
        if (rest) mine += l, before += from < lane ? l : 0;
        rest &= rest - 1;
      }
      const int at = id <= n ? tokens[id] : 0;
      if (b < B) first[b] = at + before;
      __syncwarp();
      if (b < B && lane == 31 - __clz(peers)) tokens[id] = at + mine;
      __syncwarp();
    }
  }
  __syncthreads();
  int32_t *order = a.plan + 4 + 4 * a.most;
  for (int64_t t = blockIdx.x * kThreads + tid; t < a.T; t += (int64_t)gridDim.x * kThreads) {
    if (t < all) {
      const int b = holder(cu, B, (int)t);
      order[first[b] + (int)t - cu[b]] = (int)t;
    } else {
      order[t] = -1;
    }
  }
}

constexpr size_t kMostPlanSmem = 5 * 4 * (size_t)kMostSequences;
constexpr size_t kMostGroupSmem = 4 * (size_t)(2 * kMostSequences + 1 + kMostAdapters + 1);
static_assert(kMostPlanSmem <= 224 * 1024 && kMostGroupSmem <= 224 * 1024, "the sums and counts of a CTA");

template <typename K, typename Args>
int launch_one(K kern, const Args &a, int64_t grid, int block, size_t smem, size_t most, cudaStream_t s) {
  // the limit belongs to the function, not to this call: always the largest
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e == cudaSuccess) e = launch_pdl(kern, dim3((unsigned)grid), dim3(block), smem, s, a);
  if (e != cudaSuccess) return cuda_error(e, "plan launch");
  note_launch();
  return TP_OK;
}

}  // namespace

int launch_plan(const PlanArgs &a, cudaStream_t s) {
  if (int rc = launch_one(plan_kernel, a, 1, kThreads, 5 * 4 * (size_t)a.B, kMostPlanSmem, s)) return rc;
  if (a.T <= kOwnRows) return TP_OK;
  const int64_t all = (a.T + 511) / 512, most = 4 * (int64_t)sm_count();
  return launch_one(plan_rows_kernel, a, all < most ? all : most, 512, 4 * (size_t)(a.B + 1), 4 * (kMostSequences + 1), s);
}

int launch_groups(const GroupArgs &a, cudaStream_t s) {
  const int64_t all = a.T <= kOwnRows ? 1 : (a.T + kThreads - 1) / kThreads, most = sm_count();
  return launch_one(group_kernel, a, all < most ? all : most, kThreads, 4 * (size_t)(2 * a.B + 1 + a.n + 1),
                    kMostGroupSmem, s);
}

}  // namespace tp
