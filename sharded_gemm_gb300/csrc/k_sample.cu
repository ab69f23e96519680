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
#include "sample_row.cuh"

namespace tp {
namespace {

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

template <typename T>
int launch(const SampleArgs &a, cudaStream_t s) {
  cudaError_t e;
  if (a.V > kMostOnChip) {
    // longer than a cluster holds: read again for every pass
    e = launch_pdl(sample_wide_kernel<T>, dim3((unsigned)a.B), dim3(kThreads), 0, s, a);
  } else {
    return launch_rows<T, false>(a, ctas_a_row<T, false>(a), s);
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
