// serve.cuh -- the arguments of the operators that serve many requests at once: the
// step's plan over a shared pool of pages, the grouping of its tokens by adapter, and
// the adapters' products.
#pragma once

#include "attn.cuh"

namespace tp {

constexpr int64_t kMostSequences = 8192;  // their offsets are held in shared memory
constexpr int64_t kMostAdapters = 16384;  // and the adapters' token counts

struct PlanArgs {
  const int32_t *counts, *rejected, *seq_lens, *owned, *free_count;  // rejected nullable
  int32_t *table, *free_pages;
  int32_t *new_lens, *new_owned, *new_free_count, *missing, *cu, *positions;
  int64_t *slots;
  int64_t B, width, ld_table, pages, T, cap;
  int page_log2;
  int *status;
};

// The plan of a step's adapters: a header of 4, the groups of 4, the tokens in their order.
struct GroupArgs {
  const int32_t *adapters, *cu;  // cu nullable: one token each
  int32_t *plan;
  int64_t B, T, n, most;  // most: groups there is room for
  int *status;
};
inline int64_t most_groups(int64_t T, int64_t n) { return T < n + 1 ? T : n + 1; }
inline int64_t plan_ints(int64_t T, int64_t n) { return 4 + 4 * most_groups(T, n) + T; }

// Steps of more tokens take two passes with h between them in memory; the binding asks for their
// workspace by the same rule (marshal.c).  One pass reads an adapter for every 16 tokens, the two
// for every 64 or more, but they cost a launch more.  (4096 x 4096, tokens of 8 adapters, one pass
// | two: R = 16, 1024 tokens 12.4 us | 15.0, 2048 22.7 | 18.3; R = 64, 1024 20.4 | 25.9, 2048 32.0 |
// 28.5; R = 128, 256 14.6 | 22.0, 512 24.6 | 25.8, 1024 54 | 27.  Of 250 adapters a tile holds few
// tokens either way, and up to R = 64 one pass stays ahead: 1100 tokens, R = 16 38 | 59, R = 64 61 |
// 93, R = 128 153 | 131.  The call does not know how many adapters its tokens have.)
inline int64_t few_tokens(int R) { return R <= 64 ? 1024 : 512; }
// How often a tile's contraction is split at most: few tiles leave SMs idle.
inline int lora_splits(int64_t T) { return T <= 4096 ? 8 : T <= 8192 ? 4 : T <= 16384 ? 2 : 1; }
inline int64_t lora_workspace(int64_t T, int R) {
  return T <= few_tokens(R) ? 0 : T * (R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128) * lora_splits(T);
}

struct LoraArgs {
  const void *x[kMaxShards], *a[kMaxShards];  // nx parts of the contraction
  const void *b[kMaxShards], *y[kMaxShards];  // ny parts of the output
  void *out[kMaxShards];
  const int32_t *plan;
  const float *scales;  // nullable, (n)
  int64_t T, n, K, O, ldx, ldy, ldo, most;  // K, O: of a part
  int nx, ny, R;
  int dt, out_dt;
  int in_place;  // out is y: tokens without an adapter are left alone
  float *workspace;  // many tokens: (splits, T, R rounded up to 16, 32, 64 or 128); else null
  int splits;
  int *status;
};

int launch_plan(const PlanArgs &a, cudaStream_t s);
int launch_groups(const GroupArgs &a, cudaStream_t s);
int launch_lora(const LoraArgs &a, cudaStream_t s);
int launch_lora_simt(const LoraArgs &a, cudaStream_t s);

}  // namespace tp
