// tp_attn.cu -- the C ABI of the attention-side entry points: argument checks
// and dispatch of the paged append, the paged attentions and the token draw.
#include "attn.cuh"

using namespace tp;

namespace {

bool aligned(const void *p, int a) { return ((uintptr_t)p % (uintptr_t)a) == 0; }
bool is16(int dt) { return dt == TP_BF16 || dt == TP_F16; }
int elem_size(int dt) { return dt == TP_F32 ? 4 : 2; }

int log2_of(int power) {
  int n = 0;
  while (1 << n < power) ++n;
  return n;
}

// The checks that the cache of every entry point shares.
int check_cache(int N, int Hq, int Hk, int D, int64_t pages, int page, int64_t ld_page, tp_dtype dt,
                void *const *k_cache, void *const *v_cache) {
  if (N < 1 || N > kMaxShards) return set_error(TP_ERR_INVALID_ARG, "N must be in 1..%d", kMaxShards);
  if (!is16(dt)) return set_error(TP_ERR_INVALID_ARG, "the cache holds TP_BF16 or TP_F16");
  if (Hq < 1 || Hk < 1) return set_error(TP_ERR_INVALID_ARG, "need Hq >= 1, Hk >= 1");
  if ((int64_t)Hq + 2ll * Hk > 65535)  // a launch's second dimension; N * Hq * D then fits 32 bits too
    return set_error(TP_ERR_UNSUPPORTED, "%d query and %d key-value heads: Hq + 2 Hk must be at most 65535", Hq, Hk);
  if (Hq % Hk)
    return set_error(TP_ERR_NOT_DIVISIBLE, "%d query heads cannot share %d key-value heads evenly", Hq, Hk);
  if (D != 64 && D != 128) return set_error(TP_ERR_UNSUPPORTED, "head size %d: only 64 and 128 are supported", D);
  if (page < 16 || page > 256 || (page & (page - 1)))
    return set_error(TP_ERR_UNSUPPORTED, "page size %d: must be a power of two in 16..256", page);
  if (pages < 0 || pages > 0x7fffffff) return set_error(TP_ERR_INVALID_ARG, "pages must be in 0..2^31 - 1");
  if (ld_page < (int64_t)Hk * page * D || ld_page % D)
    return set_error(TP_ERR_INVALID_ARG, "ld_page (%lld) must be a multiple of D and at least Hk * page * D",
                     (long long)ld_page);
  if (!k_cache || !v_cache) return set_error(TP_ERR_INVALID_ARG, "null pointer");
  for (int r = 0; r < N; ++r) {
    if (pages > 0 && (!k_cache[r] || !v_cache[r]))
      return set_error(TP_ERR_INVALID_ARG, "k_cache[%d] or v_cache[%d] is NULL", r, r);
    if (!aligned(k_cache[r], 16) || !aligned(v_cache[r], 16))
      return set_error(TP_ERR_ALIGNMENT, "k_cache[%d] or v_cache[%d] not 16-byte aligned", r, r);
  }
  return TP_OK;
}

int check_rows(int N, const void *const *x, int64_t ld, int64_t cols, int elem, const char *name) {
  if (!x) return set_error(TP_ERR_INVALID_ARG, "null pointer");
  if (ld < cols)
    return set_error(TP_ERR_INVALID_ARG, "row stride of %s (%lld) < its columns (%lld)", name, (long long)ld,
                     (long long)cols);
  for (int r = 0; r < N; ++r) {
    if (!x[r]) return set_error(TP_ERR_INVALID_ARG, "%s[%d] is NULL", name, r);
    if (!aligned(x[r], elem)) return set_error(TP_ERR_ALIGNMENT, "%s[%d] not aligned to its element size", name, r);
  }
  return TP_OK;
}

// The arguments that both attentions share, checked; T rows of q and o.
int attn_args(AttnArgs &a, int N, const void *const *q, int64_t T, int64_t ldq, int Hq, int Hk, int D,
              void *const *k_cache, void *const *v_cache, int64_t pages, int page, int64_t ld_page,
              const int32_t *block_table, int64_t B, int64_t width, int64_t ld_table, const int32_t *seq_lens,
              float scale, float softcap, int window, tp_dtype dt, void *const *o, int64_t ldo) {
  if (int rc = check_cache(N, Hq, Hk, D, pages, page, ld_page, dt, k_cache, v_cache)) return rc;
  if (T < 0 || B < 0 || width < 0 || T > 0x7fffffff || B > 0x7fffffff || width > 0x7fffffff)
    return set_error(TP_ERR_INVALID_ARG, "T, B and width must be in 0..2^31 - 1");
  if (T > kMostPositions) return set_error(TP_ERR_UNSUPPORTED, "T (%lld) above 2^30", (long long)T);
  if (!(scale > 0.0f) || scale > 3.0e38f) return set_error(TP_ERR_INVALID_ARG, "scale must be positive and finite");
  if (!(softcap >= 0.0f) || softcap > 3.0e38f)
    return set_error(TP_ERR_INVALID_ARG, "softcap must be finite and >= 0 (0: none)");
  if (window < 0) return set_error(TP_ERR_INVALID_ARG, "window must be >= 0 (0: none)");
  if (ld_table < width) return set_error(TP_ERR_INVALID_ARG, "ld_table < width");
  if (T > 0) {
    if (int rc = check_rows(N, q, ldq, (int64_t)Hq * D, 2, "q")) return rc;
    if (int rc = check_rows(N, o, ldo, (int64_t)Hq * D, 2, "o")) return rc;
    if (B < 1 || !seq_lens || (width > 0 && !block_table)) return set_error(TP_ERR_INVALID_ARG, "null pointer");
    if (!aligned(seq_lens, 4) || !aligned(block_table, 4))
      return set_error(TP_ERR_ALIGNMENT, "seq_lens or block_table not aligned to its element size");
  }
  memset(&a, 0, sizeof(a));
  for (int r = 0; r < N && T > 0; ++r)
    a.q[r] = q[r], a.o[r] = o[r], a.k_cache[r] = k_cache[r], a.v_cache[r] = v_cache[r];
  a.block_table = block_table, a.seq_lens = seq_lens;
  a.T = T, a.B = B, a.ldq = ldq, a.ldo = ldo, a.pages = pages, a.ld_page = ld_page;
  a.ld_table = ld_table, a.width = width;
  a.N = N, a.Hq = Hq, a.Hk = Hk, a.D = D, a.page = page;
  a.page_log2 = log2_of(page);
  const int64_t held = width << a.page_log2, most = kMostPositions;
  a.cap = held < most ? held : most;
  // a window of as many positions as there can be hides none
  a.dt = dt, a.window = window < most ? window : (int)most, a.scale = scale, a.softcap = softcap;
  return TP_OK;
}

int need_status(int **status) {
  *status = device_status_word();
  return *status ? TP_OK : set_error(TP_ERR_CUDA, "cannot allocate the device status word");
}

}  // namespace

extern "C" {

int tp_qkv_append(int N, const void *const *qkv, int64_t T, int64_t ld, tp_dtype in_dt, int Hq, int Hk, int D,
                  const float *q_norm, const float *k_norm, float eps, const float *rope, int64_t rope_rows,
                  int rope_dim, int interleaved, const int32_t *positions, const int64_t *slots, void *const *q,
                  int64_t ldq, void *const *k_cache, void *const *v_cache, int64_t pages, int page, int64_t ld_page,
                  tp_dtype dt, tp_stream_t stream) {
  if (int rc = check_cache(N, Hq, Hk, D, pages, page, ld_page, dt, k_cache, v_cache)) return rc;
  if (T < 0 || T > 0x7fffffff) return set_error(TP_ERR_INVALID_ARG, "T must be in 0..2^31 - 1");
  if (in_dt != TP_F32 && !is16(in_dt)) return set_error(TP_ERR_INVALID_ARG, "bad dtype");
  if (!(eps >= 0.0f)) return set_error(TP_ERR_INVALID_ARG, "eps must be >= 0");
  if (rope) {
    if (rope_dim < 16 || rope_dim > D || rope_dim % 16)
      return set_error(TP_ERR_UNSUPPORTED, "rope_dim %d: must be a multiple of 16 in 16..D", rope_dim);
    if (rope_rows < 1) return set_error(TP_ERR_INVALID_ARG, "need rope_rows >= 1");
  }
  if (T == 0) return TP_OK;
  if (int rc = check_rows(N, qkv, ld, (int64_t)(Hq + 2 * Hk) * D, elem_size(in_dt), "qkv")) return rc;
  if (int rc = check_rows(N, q, ldq, (int64_t)Hq * D, 2, "q")) return rc;
  if (!slots || (rope && !positions)) return set_error(TP_ERR_INVALID_ARG, "null pointer");
  if (!aligned(slots, 8) || !aligned(positions, 4) || !aligned(rope, 4) || !aligned(q_norm, 4) || !aligned(k_norm, 4))
    return set_error(TP_ERR_ALIGNMENT, "slots, positions, rope or a norm not aligned to its element size");
  AppendArgs a;
  memset(&a, 0, sizeof(a));
  for (int r = 0; r < N; ++r)
    a.qkv[r] = qkv[r], a.q[r] = q[r], a.k_cache[r] = k_cache[r], a.v_cache[r] = v_cache[r];
  a.q_norm = q_norm, a.k_norm = k_norm, a.rope = rope, a.positions = positions, a.slots = slots;
  a.T = T, a.ld = ld, a.ldq = ldq, a.pages = pages, a.ld_page = ld_page, a.rope_rows = rope_rows;
  a.N = N, a.Hq = Hq, a.Hk = Hk, a.D = D, a.page = page, a.page_log2 = log2_of(page), a.rot = rope ? rope_dim : 0, a.interleaved = interleaved != 0;
  a.in_dt = in_dt, a.dt = dt, a.eps = eps;
  if (int rc = need_status(&a.status)) return rc;
  return launch_append(a, (cudaStream_t)stream);
}

int tp_paged_decode(int N, const void *const *q, int64_t B, int64_t ldq, int Hq, int Hk, int D, void *const *k_cache,
                    void *const *v_cache, int64_t pages, int page, int64_t ld_page, const int32_t *block_table,
                    int64_t width, int64_t ld_table, const int32_t *seq_lens, float scale, float softcap, int window,
                    tp_dtype dt, void *const *o, int64_t ldo, tp_stream_t stream) {
  AttnArgs a;
  if (int rc = attn_args(a, N, q, B, ldq, Hq, Hk, D, k_cache, v_cache, pages, page, ld_page, block_table, B, width,
                         ld_table, seq_lens, scale, softcap, window, dt, o, ldo))
    return rc;
  if (B == 0) return TP_OK;
  if (int rc = need_status(&a.status)) return rc;
  return simt_policy() ? launch_attn_simt(a, (cudaStream_t)stream) : launch_decode(a, (cudaStream_t)stream);
}

int tp_paged_prefill(int N, const void *const *q, int64_t T, int64_t ldq, int Hq, int Hk, int D, void *const *k_cache,
                     void *const *v_cache, int64_t pages, int page, int64_t ld_page, const int32_t *block_table,
                     int64_t B, int64_t width, int64_t ld_table, const int32_t *cu_seqlens, const int32_t *seq_lens,
                     const int32_t *prefix_lens, float scale, float softcap, int window, tp_dtype dt, void *const *o,
                     int64_t ldo, tp_stream_t stream) {
  AttnArgs a;
  if (int rc = attn_args(a, N, q, T, ldq, Hq, Hk, D, k_cache, v_cache, pages, page, ld_page, block_table, B, width,
                         ld_table, seq_lens, scale, softcap, window, dt, o, ldo))
    return rc;
  if (T == 0) return TP_OK;
  if (!cu_seqlens) return set_error(TP_ERR_INVALID_ARG, "null pointer");
  if (!aligned(cu_seqlens, 4) || !aligned(prefix_lens, 4))
    return set_error(TP_ERR_ALIGNMENT, "cu_seqlens or prefix_lens not aligned to its element size");
  a.cu_seqlens = cu_seqlens, a.prefix_lens = prefix_lens;
  if (int rc = need_status(&a.status)) return rc;
  return simt_policy() ? launch_attn_simt(a, (cudaStream_t)stream) : launch_prefill(a, (cudaStream_t)stream);
}

int tp_sample(const void *logits, int64_t B, int64_t V, int64_t ld, tp_dtype in_dt, const float *u,
              const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p, int64_t *tokens,
              float *logprobs, tp_stream_t stream) {
  if (in_dt != TP_F32 && !is16(in_dt)) return set_error(TP_ERR_INVALID_ARG, "bad dtype");
  if (B < 0 || V < 1) return set_error(TP_ERR_INVALID_ARG, "need B >= 0, V >= 1");
  if (V > (1 << 22) || B > 0x7fffffff)
    return set_error(TP_ERR_UNSUPPORTED, "V (%lld) above 2^22 or B (%lld) above 2^31 - 1", (long long)V, (long long)B);
  if (ld < V) return set_error(TP_ERR_INVALID_ARG, "ld (%lld) < V (%lld)", (long long)ld, (long long)V);
  if (B == 0) return TP_OK;
  if (!logits || !u || !tokens) return set_error(TP_ERR_INVALID_ARG, "null pointer");
  if (!aligned(logits, elem_size(in_dt)) || !aligned(tokens, 8) || !aligned(u, 4) || !aligned(temperature, 4) ||
      !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(logprobs, 4))
    return set_error(TP_ERR_ALIGNMENT, "a pointer is not aligned to its element size");
  const SampleArgs a{logits, u, temperature, top_p, min_p, top_k, tokens, logprobs, B, V, ld, in_dt};
  return launch_sample(a, (cudaStream_t)stream);
}

}  // extern "C"
