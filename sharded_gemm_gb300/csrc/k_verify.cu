// k_verify.cu -- tp_verify: drafted tokens checked against the target's probabilities,
// from given random numbers, and the token that follows the accepted ones.
//
// With e_i, w_i and the kept prefix of a row as in tp_sample (sample_row.cuh), W the kept
// weights' total and p_i = e_i / W of the kept: drafted token d of probability q_d under
// the draft is accepted if u q_d < p_d.  Behind a sequence's accepted drafts one token is
// drawn, from max(p_i - q_i, 0) where a draft was refused, else from w: the tokens are then
// distributed as if each had been drawn from the target.  The weights of both draws are
// whole numbers of 2^-40, so their sums have no order and the token one right answer.
//
// Which row ends a sequence is known when all are done.  Every row takes its test and,
// refused, its draw at once, a cluster of CTAs each, and leaves the drawn token marked;
// a second kernel, a warp a sequence, ends the sequence at its first marked row.  (One
// cluster for the rows of a sequence, one after the other, would read no row in vain, but
// take as many times the latency as tokens were accepted.)
//
// More rows than the GPU holds are put in order first: those whose filters take several
// passes before the others, and of each kind the first rows of all sequences, then the
// second ones and so on.  A row whose sequence an earlier one has ended by then is left out.
// (436 mixed rows 155 us in the order given, all taken; 97 by their place; 92 so.  The
// ordering takes 7: rows up to 1.5 an SM go as they lie, 164 of them 60 us against 66 when that
// was chosen, 63 now.)
//
// Offsets that do not ascend are looked for by all three kernels (0.5 to 1 us in all): CTAs of a
// cluster that took a row for another sequence's would not meet at its barriers.
//
// Measured, rows of 50272: one sequence of 4 drafts 26 us; 384 rows without filters 59 (two
// turns of 152, by bytes 13); 436 with mixed settings 92 (16).
#include "sample_row.cuh"

namespace tp {
namespace {

// The order of the rows (one block): of each kind by their place in their sequences up to
// kLevels, then the others as they lie.
constexpr int kLevels = 32;
__global__ void __launch_bounds__(kThreads) verify_order_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ uint64_t sums[32];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t first = a.cu[0], end = a.cu[a.seqs];  // rows of no sequence are not touched
  int64_t r0 = 0, n = 0;
  bool slow = false, bad = false;
  auto look = [&](int64_t s) {
    n = 0;
    if (s >= a.seqs) return;
    r0 = a.cu[s];
    const int64_t r1 = a.cu[s + 1];
    if (ascend(a, r0, r1)) n = r1 - r0;
    else bad = true;
    slow = slow_row(a, s);
  };
  // the sums over lower threads of two values, side by side, and over all
  auto scan = [&](uint64_t v, uint64_t &all) {
    uint64_t run = v;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
      const uint64_t o = __shfl_up_sync(0xffffffffu, run, m);
      if (lane >= m) run += o;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = run;
    __syncthreads();
    uint64_t lower = lane < warp ? sums[lane] : 0;
    all = sums[lane];
#pragma unroll
    for (int m = 16; m > 0; m /= 2) {
      lower += __shfl_xor_sync(0xffffffffu, lower, m);
      all += __shfl_xor_sync(0xffffffffu, all, m);
    }
    return lower + run - v;
  };
  int64_t at[2] = {0, 0};  // where the next row of a slow sequence goes, and of another
  uint64_t all;
  for (int64_t base = 0; base < a.seqs; base += kThreads) {
    look(base + tid);
    scan(slow ? (uint64_t)n : 0, all);
    at[1] += (int64_t)all;
  }
  if (__syncthreads_or(bad)) return;  // the rows go as they lie
  for (int64_t i = first + tid; i < end; i += kThreads) row_words(a, i)[0] = kPending;
  auto put = [&](int64_t at, int64_t row) { row_words(a, first + at)[1] = (int32_t)row; };
  for (int level = 0; level <= kLevels; ++level) {
    bool more = false;
    for (int64_t base = 0; base < a.seqs; base += kThreads) {
      if (a.seqs > kThreads) look(base + tid);
      const uint64_t left = n > level ? n - level : 0, count = level < kLevels ? left > 0 : left;
      const uint64_t before = scan(slow ? count << 32 : count, all);
      const int64_t place = slow ? at[0] + (int64_t)(before >> 32) : at[1] + (int64_t)(before & 0xffffffffu);
      for (uint64_t i = 0; i < count; ++i) put(place + i, r0 + level + i);
      at[0] += (int64_t)(all >> 32), at[1] += (int64_t)(all & 0xffffffffu);
      more = more || left > 1;
    }
    if (!__syncthreads_or(more)) break;
  }
}

__global__ void __launch_bounds__(256) verify_end_kernel(const __grid_constant__ VerifyArgs a) {
  griddep_wait();
  const int64_t b = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int64_t r0 = b < a.seqs ? a.cu[b] : 0, r1 = b < a.seqs ? a.cu[b + 1] : 0;
  // (the first results are asked for before it is known that all offsets ascend)
  const int32_t begin = ascend(a, r0, r1) && r0 + lane < r1 ? row_words(a, r0 + lane)[0] : 0;
  bool bad = false;
  for (int64_t s = threadIdx.x; s < a.seqs; s += 256) bad = bad || !ascend(a, a.cu[s], a.cu[s + 1]);
  bad = __syncthreads_or(bad);
  if (bad && blockIdx.x == 0 && threadIdx.x == 0) record_bad_value(a.status);
  if (b >= a.seqs) return;
  int64_t accepted = 0, n = r1 - r0;
  // rows that another sequence claims are no one's
  if (!ascend(a, r0, r1) || n == 0 || (bad && __any_sync(0xffffffffu, reached(a, b, lane, 32)))) {
    n = 1;
  } else {
    bool ended = false;
    for (int64_t i0 = r0; i0 < r1; i0 += 32) {
      const int64_t i = i0 + lane;
      const int32_t word = i0 == r0 ? begin : i < r1 ? row_words(a, i)[0] : 0;
      const uint32_t marked = __ballot_sync(0xffffffffu, i < r1 && word < 0);
      const int end = ended ? -1 : marked ? __ffs(marked) - 1 : 32;
      if (i < r1) a.tokens[i] = lane < end ? word : lane == end ? drawn_mark(word) : -1;
      if (i < r1 && lane > end && a.logprobs) a.logprobs[i] = 0.0f;
      if (!ended && marked) accepted = i0 + end - r0, ended = true;
    }
  }
  if (lane == 0) {
    if (a.accepted) a.accepted[b] = (int32_t)accepted;
    if (a.rejected) a.rejected[b] = (int32_t)(n - 1 - accepted);
  }
}

static_assert(kMostVerified == kMostOnChip, "the argument check");

template <typename T>
int launch(VerifyArgs a, cudaStream_t s) {
  cudaError_t e;
  if (a.B > 0) {
    const int C = ctas_a_row<T, true>(a);
    a.ordered = a.B * C > 3 * sm_count() / 2;
    if (a.ordered) {
      e = launch_pdl(verify_order_kernel, dim3(1), dim3(kThreads), 0, s, a);
      if (e != cudaSuccess) return cuda_error(e, "verify launch");
      note_launch();
    }
    if (int rc = launch_rows<T, true>(a, C, s)) return rc;
  }
  e = launch_pdl(verify_end_kernel, dim3((unsigned)((a.seqs + 7) / 8)), dim3(256), 0, s, a);
  if (e != cudaSuccess) return cuda_error(e, "verify launch");
  note_launch();
  return TP_OK;
}

}  // namespace

int launch_verify(const VerifyArgs &a, cudaStream_t s) {
  if (a.in_dt == TP_F32) return launch<float>(a, s);
  return a.in_dt == TP_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

}  // namespace tp
