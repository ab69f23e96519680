// k_attn_simt.cu -- paged attention on the CUDA cores: one warp per query row
// and head, 32 keys at a time with the running maximum and sum of a softmax.
// The slow cross-check of the tensor-core kernels (TP_POLICY_SIMT), for one
// token per sequence (cu_seqlens null) and for ragged chunks alike.
#include "attn.cuh"
#include "ptx.cuh"

namespace tp {
namespace {

constexpr int kWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) attn_simt_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int E = D / 32;
  __shared__ float sq[kWarps][D];
  griddep_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t rows = a.T * a.N * a.Hq;
  if (a.cu_seqlens && lane == 0)
    for (int64_t i = w; i < a.B; i += (int64_t)gridDim.x * kWarps) {
      const int c0 = a.cu_seqlens[i], c1 = a.cu_seqlens[i + 1];
      if (c0 < 0 || c1 < c0 || c1 > a.T) record_bad_value(a.status);
    }
  if (w >= rows) return;
  const int hq = (int)(w % a.Hq);
  const int r = (int)(w / a.Hq % a.N);
  const int64_t t = w / ((int64_t)a.Hq * a.N);
  const int h = hq / (a.Hq / a.Hk);
  T *out = static_cast<T *>(a.o[r]) + t * a.ldo + (int64_t)hq * D;

  // the row's sequence and its place in it
  int64_t b = t, pos, first = 0, n = 0;
  if (a.cu_seqlens) {
    int64_t lo = 0, hi = a.B;  // the last b with cu[b] <= t
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) / 2;
      if (a.cu_seqlens[mid] <= t) lo = mid; else hi = mid;
    }
    b = lo;
    n = a.seq_lens[b];
    pos = n - a.cu_seqlens[b + 1] + t;
    if (t < a.cu_seqlens[b] || t >= a.cu_seqlens[b + 1]) n = 0;  // a token of no sequence
  } else {
    n = a.seq_lens[b];
    pos = n - 1;
  }
  if (n < 0 || n > a.cap) {
    n = n < 0 ? 0 : a.cap;
    if (lane == 0) record_bad_value(a.status);
  }
  const int64_t prefix = a.prefix_lens ? a.prefix_lens[b] : 0;
  if (a.window && pos - a.window + 1 > 0) first = pos - a.window + 1;
  const int64_t from = prefix > 0 ? 0 : first;
  int64_t to = pos + 1 > prefix ? pos + 1 : prefix;
  if (to > n) to = n;

  const T *q = static_cast<const T *>(a.q[r]) + t * a.ldq + (int64_t)hq * D;
#pragma unroll
  for (int e = 0; e < E; ++e) sq[warp][lane + 32 * e] = static_cast<float>(q[lane + 32 * e]) * a.scale;
  __syncwarp();

  float m = -INFINITY, l = 0.0f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
  for (int64_t j0 = from & ~(int64_t)31; j0 < to; j0 += 32) {
    const int64_t j = j0 + lane;
    bool seen = j < to && ((j >= first && j <= pos) || j < prefix);
    float s = -INFINITY;
    int64_t row = 0;
    if (seen) {
      const int pg = a.block_table[b * a.ld_table + j / a.page];
      if (pg < 0 || pg >= a.pages) {
        seen = false;
        record_bad_value(a.status);
      } else {
        row = pg * a.ld_page + ((int64_t)h * a.page + j % a.page) * D;
        const uint4 *k = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.k_cache[r]) + row);
        float dot = 0.0f;
        for (int c = 0; c < D / 8; ++c) {
          const uint4 x = k[c];
          const uint32_t p[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = Half2<T>::unpack(p[i]);
            dot = fmaf(f.x, sq[warp][8 * c + 2 * i], dot);
            dot = fmaf(f.y, sq[warp][8 * c + 2 * i + 1], dot);
          }
        }
        s = a.softcap > 0.0f ? a.softcap * tanhf(dot / a.softcap) : dot;
      }
    }
    const uint32_t any = __ballot_sync(0xffffffffu, seen);
    if (!any) continue;
    float top = s;
#pragma unroll
    for (int x = 16; x > 0; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float mn = fmaxf(m, top), ms = mn == -INFINITY ? 0.0f : mn;
    const float keep = expf(m - ms);
    const float p = seen ? expf(s - ms) : 0.0f;
    float sum = p;
#pragma unroll
    for (int x = 16; x > 0; x /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = l * keep + sum;
    m = mn;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= keep;
    for (int i = 0; i < 32; ++i) {
      if (!(any >> i & 1)) continue;  // a hidden key's value is never read
      const float pi = __shfl_sync(0xffffffffu, p, i);
      const int64_t ri = __shfl_sync(0xffffffffu, row, i);
      const T *v = static_cast<const T *>(a.v_cache[r]) + ri;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(pi, static_cast<float>(v[lane + 32 * e]), acc[e]);
    }
  }
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;  // a row that sees no key is zero
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane + 32 * e] = static_cast<T>(acc[e] * inv);
}

template <typename T>
int launch(const AttnArgs &a, cudaStream_t s) {
  const int64_t blocks = (a.T * a.N * a.Hq + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffff) return set_error(TP_ERR_UNSUPPORTED, "T * N * Hq too large for one launch");
  const dim3 grid((unsigned)blocks), block(kWarps * 32);
  const cudaError_t e = a.D == 64 ? launch_pdl(attn_simt_kernel<T, 64>, grid, block, 0, s, a)
                                  : launch_pdl(attn_simt_kernel<T, 128>, grid, block, 0, s, a);
  if (e != cudaSuccess) return cuda_error(e, "attention launch");
  note_launch();
  return TP_OK;
}

}  // namespace

int launch_attn_simt(const AttnArgs &a, cudaStream_t s) {
  return a.dt == TP_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

}  // namespace tp
