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
#include "sample_row.cuh"

namespace tp {
namespace {

__global__ void __launch_bounds__(256) verify_end_kernel(const __grid_constant__ VerifyArgs a) {
  griddep_wait();
  const int64_t b = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (b >= a.seqs) return;
  const int64_t r0 = a.cu[b], r1 = a.cu[b + 1];
  int64_t accepted = 0, n = r1 - r0;
  if (r0 < 0 || n <= 0 || r1 > a.B) {
    n = 1;
  } else {
    bool ended = false;
    for (int64_t i0 = r0; i0 < r1; i0 += 32) {
      const int64_t i = i0 + lane, token = i < r1 ? a.tokens[i] : 0;
      const uint32_t marked = __ballot_sync(0xffffffffu, i < r1 && token < 0);
      const int end = ended ? -1 : marked ? __ffs(marked) - 1 : 32;
      if (i < r1 && lane == end) a.tokens[i] = drawn_mark(token);
      if (i < r1 && lane > end) {
        a.tokens[i] = -1;
        if (a.logprobs) a.logprobs[i] = 0.0f;
      }
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
int launch(const VerifyArgs &a, cudaStream_t s) {
  if (a.B > 0)
    if (int rc = launch_rows<T, true>(a, s)) return rc;
  const cudaError_t e = launch_pdl(verify_end_kernel, dim3((unsigned)((a.seqs + 7) / 8)), dim3(256), 0, s, a);
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
