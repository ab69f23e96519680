// tp_serve.cu -- the C ABI of the operators that serve many requests at once: argument
// checks and dispatch of the step's plan, the adapters and the verification of drafts.
#include "serve.cuh"

using namespace tp;

namespace {

bool aligned(const void *p, int a) { return ((uintptr_t)p % (uintptr_t)a) == 0; }
bool is16(int dt) { return dt == TP_BF16 || dt == TP_F16; }
int elem_size(int dt) { return dt == TP_F32 ? 4 : 2; }
constexpr int64_t kMost32 = 0x7fffffff;

int need_status(int **status) {
  *status = device_status_word();
  return *status ? TP_OK : set_error(TP_ERR_CUDA, "cannot allocate the device status word");
}

int check_rows(int n, const void *const *x, int64_t T, int64_t ld, int64_t cols, int elem, const char *name) {
  if (!x) return set_error(TP_ERR_INVALID_ARG, "null pointer");
  if (T > 1 && ld < cols)
    return set_error(TP_ERR_INVALID_ARG, "row stride of %s (%lld) < its columns (%lld)", name, (long long)ld,
                     (long long)cols);
  for (int r = 0; r < n; ++r) {
    if (!x[r]) return set_error(TP_ERR_INVALID_ARG, "%s[%d] is NULL", name, r);
    if (!aligned(x[r], elem)) return set_error(TP_ERR_ALIGNMENT, "%s[%d] not aligned to its element size", name, r);
  }
  return TP_OK;
}

int check_ranks(int N) {
  return N < 1 || N > kMaxShards ? set_error(TP_ERR_INVALID_ARG, "N must be in 1..%d", kMaxShards) : TP_OK;
}

int check_widths(int64_t K, int64_t O) {
  if (K < 1 || O < 1) return set_error(TP_ERR_INVALID_ARG, "need K >= 1, O >= 1");
  if (K > 1 << 30 || O > 1 << 30)  // counted in 32 bits, a block of 32 behind the end too
    return set_error(TP_ERR_UNSUPPORTED, "K (%lld) and O (%lld) must be at most 2^30", (long long)K, (long long)O);
  return TP_OK;
}

// K and O those of a part.
int lora(int nx, const void *const *x, int64_t T, int64_t K, int64_t ldx, const void *const *a, int ny,
         const void *const *b, int64_t n, int R, int64_t O, const float *scales, const int32_t *plan,
         int64_t plan_size, float *workspace, tp_dtype dt, const void *const *y, int64_t ldy, void *const *out,
         int64_t ldo, tp_dtype out_dt, tp_stream_t stream) {
  if (!is16(dt)) return set_error(TP_ERR_INVALID_ARG, "the adapters hold TP_BF16 or TP_F16");
  if (out_dt != TP_F32 && !is16(out_dt)) return set_error(TP_ERR_INVALID_ARG, "bad dtype");
  if (T < 0 || T > kMost32 || n < 1) return set_error(TP_ERR_INVALID_ARG, "need T in 0..2^31 - 1, n >= 1");
  if (n > kMostAdapters)
    return set_error(TP_ERR_UNSUPPORTED, "%lld adapters: at most %lld", (long long)n, (long long)kMostAdapters);
  if (R < 1) return set_error(TP_ERR_INVALID_ARG, "need R >= 1");
  if (R > 128) return set_error(TP_ERR_UNSUPPORTED, "rank %d: at most 128", R);
  if (T == 0) return TP_OK;
  const int es = elem_size(out_dt);
  if (int rc = check_rows(nx, x, T, ldx, K, 2, "x")) return rc;
  if (int rc = check_rows(nx, a, 0, K, K, 2, "a")) return rc;
  if (int rc = check_rows(ny, b, 0, R, R, 2, "b")) return rc;
  if (int rc = check_rows(ny, y, T, ldy, O, es, "y")) return rc;
  if (int rc = check_rows(ny, out, T, ldo, O, es, "out")) return rc;
  if (!plan) return set_error(TP_ERR_INVALID_ARG, "null pointer");
  if (!aligned(plan, 16) || !aligned(workspace, 16) || !aligned(scales, 4))
    return set_error(TP_ERR_ALIGNMENT, "plan or workspace not aligned to 16 bytes, or scales not to 4");
  if (plan_size != plan_ints(T, n))
    return set_error(TP_ERR_INVALID_ARG, "a plan of %lld values: %lld rows and %lld adapters have %lld",
                     (long long)plan_size, (long long)T, (long long)n, (long long)plan_ints(T, n));
  LoraArgs l;
  memset(&l, 0, sizeof(l));
  for (int r = 0; r < nx; ++r) l.x[r] = x[r], l.a[r] = a[r];
  int same = 0;
  for (int r = 0; r < ny; ++r) {
    l.b[r] = b[r], l.y[r] = y[r], l.out[r] = out[r];
    same += y[r] == out[r];
  }
  if (same && (same < ny || (T > 1 && ldy != ldo)))
    return set_error(TP_ERR_INVALID_ARG, "out must be y for all ranks, with one row stride, or for none");
  l.plan = plan, l.scales = scales, l.workspace = lora_workspace(T, R) > 0 ? workspace : nullptr, l.splits = lora_splits(T);
  l.T = T, l.n = n, l.K = K, l.O = O, l.ldx = ldx, l.ldy = ldy, l.ldo = ldo, l.most = most_groups(T, n);
  l.nx = nx, l.ny = ny, l.R = R, l.dt = dt, l.out_dt = out_dt, l.in_place = same != 0;
  if (int rc = need_status(&l.status)) return rc;
  return simt_policy() ? launch_lora_simt(l, (cudaStream_t)stream) : launch_lora(l, (cudaStream_t)stream);
}

}  // namespace

extern "C" {

int tp_paged_plan(int64_t B, const int32_t *counts, const int32_t *rejected, const int32_t *seq_lens,
                  const int32_t *owned, int32_t *block_table, int64_t width, int64_t ld_table, int32_t *free_pages,
                  int64_t pages, const int32_t *free_count, int page, int64_t T, int32_t *new_seq_lens,
                  int32_t *new_owned, int32_t *new_free_count, int32_t *missing, int32_t *cu_seqlens,
                  int32_t *positions, int64_t *slots, tp_stream_t stream) {
  if (B < 0 || T < 0 || T > kMost32 || width < 0 || width > kMost32 || pages < 0 || pages > kMost32)
    return set_error(TP_ERR_INVALID_ARG, "B, T, width and pages must be in 0..2^31 - 1");
  if (B > kMostSequences)
    return set_error(TP_ERR_UNSUPPORTED, "%lld sequences: at most %lld", (long long)B, (long long)kMostSequences);
  if (page < 16 || page > 256 || (page & (page - 1)))
    return set_error(TP_ERR_UNSUPPORTED, "page size %d: must be a power of two in 16..256", page);
  if (ld_table < width) return set_error(TP_ERR_INVALID_ARG, "ld_table < width");
  if ((B > 0 && (!counts || !seq_lens || !owned || !new_seq_lens || !new_owned || (width > 0 && !block_table))) ||
      (pages > 0 && !free_pages) || !free_count || !new_free_count || !missing || !cu_seqlens ||
      (T > 0 && (!positions || !slots)))
    return set_error(TP_ERR_INVALID_ARG, "null pointer");
  const void *words[] = {counts, rejected, seq_lens, owned, block_table, free_pages, free_count, new_seq_lens,
                         new_owned, new_free_count, missing, cu_seqlens, positions};
  for (const void *w : words)
    if (!aligned(w, 4)) return set_error(TP_ERR_ALIGNMENT, "a pointer is not aligned to its element size");
  if (!aligned(slots, 8)) return set_error(TP_ERR_ALIGNMENT, "a pointer is not aligned to its element size");
  PlanArgs a;
  memset(&a, 0, sizeof(a));
  a.counts = counts, a.rejected = rejected, a.seq_lens = seq_lens, a.owned = owned, a.free_count = free_count;
  a.table = block_table, a.free_pages = free_pages;
  a.new_lens = new_seq_lens, a.new_owned = new_owned, a.new_free_count = new_free_count, a.missing = missing;
  a.cu = cu_seqlens, a.positions = positions, a.slots = slots;
  a.B = B, a.width = width, a.ld_table = ld_table, a.pages = pages, a.T = T;
  while (1 << a.page_log2 < page) ++a.page_log2;
  const int64_t held = width << a.page_log2;
  a.cap = held < kMostPositions ? held : kMostPositions;
  if (int rc = need_status(&a.status)) return rc;
  return launch_plan(a, (cudaStream_t)stream);
}

int64_t tp_lora_plan_ints(int64_t T, int64_t n) { return T < 0 || n < 0 ? 0 : plan_ints(T, n); }

int64_t tp_lora_workspace_floats(int64_t T, int R) { return T < 0 || R < 1 || R > 128 ? 0 : lora_workspace(T, R); }

int tp_lora_plan(int64_t B, const int32_t *adapters, const int32_t *cu_seqlens, int64_t T, int64_t n, int32_t *plan,
                 tp_stream_t stream) {
  if (B < 0 || T < 0 || T > kMost32 || n < 1) return set_error(TP_ERR_INVALID_ARG, "need B >= 0, T >= 0, n >= 1");
  if (B > kMostSequences || n > kMostAdapters)
    return set_error(TP_ERR_UNSUPPORTED, "%lld sequences, %lld adapters: at most %lld and %lld", (long long)B,
                     (long long)n, (long long)kMostSequences, (long long)kMostAdapters);
  if (!cu_seqlens && B != T) return set_error(TP_ERR_INVALID_ARG, "without cu_seqlens B must be T");
  if (!plan || (B > 0 && !adapters)) return set_error(TP_ERR_INVALID_ARG, "null pointer");
  if (!aligned(plan, 16) || !aligned(adapters, 4) || !aligned(cu_seqlens, 4))
    return set_error(TP_ERR_ALIGNMENT, "plan not aligned to 16 bytes, or an array not to its element size");
  GroupArgs a;
  memset(&a, 0, sizeof(a));
  a.adapters = adapters, a.cu = cu_seqlens, a.plan = plan, a.B = B, a.T = T, a.n = n, a.most = most_groups(T, n);
  if (int rc = need_status(&a.status)) return rc;
  return launch_groups(a, (cudaStream_t)stream);
}

int tp_lora_all_to_sharded(int N, const void *x, int64_t T, int64_t K, int64_t ldx, const void *a,
                           const void *const *b, int64_t n, int R, int64_t O, const float *scales,
                           const int32_t *plan, int64_t plan_size, float *workspace, tp_dtype dt,
                           const void *const *y, int64_t ldy, void *const *out, int64_t ldo, tp_dtype out_dt,
                           tp_stream_t stream) {
  if (int rc = check_ranks(N)) return rc;
  if (int rc = check_widths(K, O)) return rc;
  if (O % N) return set_error(TP_ERR_NOT_DIVISIBLE, "Cannot shard %lld outputs over %d ranks", (long long)O, N);
  return lora(1, &x, T, K, ldx, &a, N, b, n, R, O / N, scales, plan, plan_size, workspace, dt, y, ldy, out, ldo, out_dt,
              stream);
}

int tp_lora_sharded_to_all(int N, const void *const *x, int64_t T, int64_t K, int64_t ldx, const void *const *a,
                           const void *b, int64_t n, int R, int64_t O, const float *scales, const int32_t *plan,
                           int64_t plan_size, float *workspace, tp_dtype dt, const void *y, int64_t ldy, void *out,
                           int64_t ldo, tp_dtype out_dt, tp_stream_t stream) {
  if (int rc = check_ranks(N)) return rc;
  if (int rc = check_widths(K, O)) return rc;
  if (K % N) return set_error(TP_ERR_NOT_DIVISIBLE, "Cannot shard %lld inputs over %d ranks", (long long)K, N);
  return lora(N, x, T, K / N, ldx, a, 1, &b, n, R, O, scales, plan, plan_size, workspace, dt, &y, ldy, &out, ldo,
              out_dt, stream);
}

int tp_verify(const void *logits, int64_t T, int64_t V, int64_t ld, tp_dtype in_dt, const int64_t *drafts,
              const void *draft_probs, int64_t ldq, tp_dtype q_dt, int64_t seqs, const int32_t *cu_rows, const float *u,
              const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p, int64_t *tokens,
              float *logprobs, int32_t *accepted, int32_t *rejected, tp_stream_t stream) {
  if ((in_dt != TP_F32 && !is16(in_dt)) || (draft_probs && q_dt != TP_F32 && !is16(q_dt)))
    return set_error(TP_ERR_INVALID_ARG, "bad dtype");
  if (T < 0 || V < 1 || seqs < 0) return set_error(TP_ERR_INVALID_ARG, "need T >= 0, V >= 1, seqs >= 0");
  if (T > kMost32 / 8 || seqs > kMost32 / 8)
    return set_error(TP_ERR_UNSUPPORTED, "T (%lld) or seqs (%lld) above 2^28 - 1", (long long)T, (long long)seqs);
  if (V > kMostVerified)
    return set_error(TP_ERR_UNSUPPORTED, "V (%lld): at most %lld", (long long)V, (long long)kMostVerified);
  if (ld < V || (draft_probs && ldq < V)) return set_error(TP_ERR_INVALID_ARG, "a row stride is below V (%lld)", (long long)V);
  if (seqs == 0) return TP_OK;
  if (!cu_rows || (T > 0 && (!logits || !drafts || !u || !tokens))) return set_error(TP_ERR_INVALID_ARG, "null pointer");
  if (!aligned(logits, elem_size(in_dt)) || !aligned(draft_probs, elem_size(q_dt)) || !aligned(drafts, 8) ||
      !aligned(tokens, 8) || !aligned(cu_rows, 4) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
      !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(logprobs, 4) || !aligned(accepted, 4) || !aligned(rejected, 4))
    return set_error(TP_ERR_ALIGNMENT, "a pointer is not aligned to its element size");
  VerifyArgs a;
  memset(&a, 0, sizeof(a));
  a.logits = logits, a.u = u, a.temperature = temperature, a.top_p = top_p, a.min_p = min_p, a.top_k = top_k;
  a.tokens = tokens, a.logprobs = logprobs, a.B = T, a.V = V, a.ld = ld, a.in_dt = in_dt;
  a.cu = cu_rows, a.drafts = drafts, a.q = draft_probs, a.accepted = accepted, a.rejected = rejected;
  a.seqs = seqs, a.ldq = ldq, a.q_dt = q_dt;
  if (int rc = need_status(&a.status)) return rc;
  return launch_verify(a, (cudaStream_t)stream);
}

}  // extern "C"
