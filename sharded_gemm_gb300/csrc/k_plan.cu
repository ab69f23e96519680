// k_plan.cu -- tp_paged_plan and tp_lora_plan: what a serving step needs to know of its
// tokens, built from the requests' lengths on the GPU.
//
// tp_paged_plan.  Three running sums over the sequences (tokens, pages that ended ones
// give back, pages needed) place everything: token i of sequence b in row cu[b] + i, the
// i-th page given back on top of the pool, the i-th page needed taken from the top.  One
// cluster does it in one launch: every CTA reads the sequences and takes the sums for
// itself, a barrier lies between that and the first write (outputs may be the inputs
// themselves), and the rows and pages are dealt to the threads of all CTAs, each of which
// finds its sequence by bisection of the sums in shared memory.
//
// tp_lora_plan.  A stable counting sort by adapter: tokens of each adapter counted in
// shared memory, their running sum, and then one warp walks the sequences in order, 32 at
// a time, and gives each the place behind the earlier ones of its adapter.  The tokens are
// then dealt to all threads.  Every CTA of the cluster does the counting for itself.
//
// Both are bound by latency: two or three dependent loads, the sums' barriers, the
// bisections.  A step of few tokens takes one CTA.
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

__global__ void __launch_bounds__(kThreads) plan_kernel(const __grid_constant__ PlanArgs a, int C) {
  extern __shared__ int32_t smem[];
  __shared__ int64_t buf[96];
  const int B = (int)a.B, tid = threadIdx.x, rank = blockIdx.x;
  int32_t *cu = smem, *need_at = cu + B, *back_at = need_at + B, *after = back_at + B, *held = after + B;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t F = a.free_count[0], page = 1ll << a.page_log2;

  // ---- a run of sequences a thread, and the sums before them
  const int run = (B + kThreads - 1) / kThreads, b0 = tid * run, b1 = min(b0 + run, B);
  bool bad = F < 0 || F > a.pages;
  int64_t sums[3] = {0, 0, 0}, total[3];
  auto sequence = [&](int b, int64_t &tokens, int64_t &need, int64_t &back, int64_t &end, int64_t &own) {
    const int64_t c = a.counts[b], len = a.seq_lens[b], less = a.rejected ? a.rejected[b] : 0;
    own = a.owned[b];
    tokens = need = back = end = 0;
    if (own < 0 || own > a.width) return false;
    if (c < 0) {
      back = own;
      return true;
    }
    end = len - less + c, tokens = c;
    const int64_t pages = (end + page - 1) >> a.page_log2;
    need = pages > own ? pages - own : 0;
    return len >= 0 && less >= 0 && less <= len && end <= a.cap && (own << a.page_log2) >= len - less;
  };
  for (int b = b0; b < b1; ++b) {
    int64_t tokens, need, back, end, own;
    if (sequence(b, tokens, need, back, end, own)) sums[0] += tokens, sums[1] += need, sums[2] += back;
    else bad = true;
  }
  scan_before<3>(sums, total, buf);
  const int64_t top = F + total[2];  // of the pool, what ended sequences give back on it
  bad = __syncthreads_or(bad) || top > a.pages || total[0] > a.T;
  const bool fits = !bad && total[1] <= top;
  for (int b = b0; b < b1; ++b) {
    int64_t tokens, need, back, end, own;
    sequence(b, tokens, need, back, end, own);
    if (!fits) end = a.seq_lens[b];  // an empty step
    cu[b] = fits ? (int32_t)sums[0] : 0, need_at[b] = (int32_t)sums[1], back_at[b] = (int32_t)sums[2];
    after[b] = (int32_t)end, held[b] = a.owned[b];
    sums[0] += tokens, sums[1] += need, sums[2] += back;
  }
  const int total_tokens = fits ? (int)total[0] : 0, total_need = fits ? (int)total[1] : 0;
  const int total_back = fits ? (int)total[2] : 0;
  // every CTA has read what is overwritten below, and the sums are in shared memory
  if (C > 1) cluster_sync_all(); else __syncthreads();

  const int thread = rank * kThreads + tid, threads = C * kThreads;
  for (int b = thread; b < B; b += threads) {
    const int own = held[b], all = b + 1 < B ? need_at[b + 1] : (int)total[1];
    const bool ends = fits && (b + 1 < B ? back_at[b + 1] : total_back) > back_at[b];
    a.cu[b] = cu[b];
    a.new_lens[b] = after[b];
    // (a sequence that ended with no pages has none to need either)
    a.new_owned[b] = !fits ? own : ends ? 0 : own + (all - need_at[b]);
  }
  if (thread == 0) {
    a.cu[B] = total_tokens;
    a.new_free_count[0] = fits ? (int32_t)(top - total[1]) : (int32_t)F;
    a.missing[0] = bad ? -1 : fits ? 0 : (int32_t)(total[1] - top);
    if (bad) record_bad_value(a.status);
  }
  // ---- pages given back go on top of the pool
  for (int i = thread; i < total_back; i += threads) {
    const int b = holder(back_at, B, i);
    a.free_pages[F + i] = a.table[b * a.ld_table + (i - back_at[b])];
  }
  if (total_back > 0 && total_need > 0) {  // the same in all CTAs
    __threadfence();
    if (C > 1) cluster_sync_all(); else __syncthreads();
  }
  // ---- and what is needed is taken from there
  auto taken = [&](int i) { return __ldcg(a.free_pages + (top - 1 - i)); };
  for (int i = thread; i < total_need; i += threads) {
    const int b = holder(need_at, B, i);
    a.table[b * a.ld_table + held[b] + (i - need_at[b])] = taken(i);
  }
  // ---- the tokens: pages taken just now are read from the pool
  for (int64_t t = thread; t < a.T; t += threads) {
    int32_t position = 0;
    int64_t slot = -1;
    if (t < total_tokens) {
      const int b = holder(cu, B, (int)t), end = b + 1 < B ? cu[b + 1] : total_tokens;
      position = after[b] - (end - (int)t);
      const int j = position >> a.page_log2;
      const int32_t p = j < held[b] ? a.table[b * a.ld_table + j] : taken(need_at[b] + j - held[b]);
      if (p >= 0 && p < a.pages) slot = ((int64_t)p << a.page_log2) + (position & (int)(page - 1));
      else record_bad_value(a.status);
    }
    a.positions[t] = position;
    a.slots[t] = slot;
  }
}

__global__ void __launch_bounds__(kThreads) group_kernel(const __grid_constant__ GroupArgs a, int C) {
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
      int before = 0, mine = 0;
      for (int i = 0; i < 32; ++i) {
        const int l = __shfl_sync(0xffffffffu, len, i);
        if (peers >> i & 1) {
          mine += l;
          if (i < lane) before += l;
        }
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
  for (int64_t t = blockIdx.x * kThreads + tid; t < a.T; t += C * kThreads) {
    if (t < all) {
      const int b = holder(cu, B, (int)t);
      order[first[b] + (int)t - cu[b]] = (int)t;
    } else {
      order[t] = -1;
    }
  }
}

// One cluster: a CTA for few rows, else eight.  (A cluster's launch and barriers cost about
// 2 us more than one CTA's; 4096 rows are four turns of a CTA's threads.)
template <typename Args>
int launch_cluster(void (*kern)(Args, int), const Args &a, int64_t rows, size_t smem, cudaStream_t s,
                   const char *what) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (e != cudaSuccess) return cuda_error(e, what);
  const int C = rows > 4096 ? 8 : 1;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(C);
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
  e = cudaLaunchKernelEx(&cfg, kern, a, C);
  if (e != cudaSuccess) return cuda_error(e, what);
  note_launch();
  return TP_OK;
}

static_assert(5 * 4 * kMostSequences <= 200 * 1024, "plan_kernel's sums");
static_assert(4 * (2 * kMostSequences + 1 + kMostAdapters + 1) <= 200 * 1024, "group_kernel's counts");

}  // namespace

int launch_plan(const PlanArgs &a, cudaStream_t s) {
  return launch_cluster(plan_kernel, a, a.T, 5 * 4 * (size_t)a.B, s, "plan launch");
}

int launch_groups(const GroupArgs &a, cudaStream_t s) {
  return launch_cluster(group_kernel, a, a.T, 4 * (size_t)(2 * a.B + 1 + a.n + 1), s, "adapter plan launch");
}

}  // namespace tp
